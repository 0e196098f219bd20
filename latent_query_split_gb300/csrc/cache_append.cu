// cache_append.cu -- new tokens enter the paged 8-bit cache, keys (and queries)
// rotated by their positions on the way.
//
// Rotation of channel pair j at position p by the angle a = p * inv_freq[j]:
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a).
// The angle is taken in turns as a 64-bit binary fraction: f = inv_freq / 2 pi
// mod 1 in units of 2^-64, so that p * f mod 2^64 is the angle mod one turn,
// within 2^-32 at any position; its top 32 bits go to sincospi.
//
// Codes of a page and head share a scale 2^e, -40 <= e <= 60. With A the
// largest magnitude of the new tokens (before the rotation), A 2^-e lies in
// (128, 256]; the rotation lengthens one channel at most sqrt(2) times, which
// leaves 362 < 448, so nothing saturates and the scale does not hang on the
// rotation's roundings. A power of two costs an e4m3 code no precision. A page
// that holds earlier tokens of the sequence keeps the larger of both scales;
// where that is the new one, the old codes are rescaled (a shift of their
// exponents: exact but for codes that become subnormal).
#include "cache_common.cuh"

#include <cuda_fp8.h>

namespace flare {
namespace cache {
namespace {

constexpr int kEMin = -40, kEMax = 60;

__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// ceil(log2 a) - 8, clamped; a = 0 (or subnormal) takes the lowest.
__device__ __forceinline__ int exponent_of(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 + ((u & 0x7fffffu) ? 1 : 0) - 8;
    return u < 0x00800000u ? kEMin : imax(kEMin, imin(kEMax, e));
}
// The exponent of a stored scale; what is no power of two in range is taken
// for the nearest one below.
__device__ __forceinline__ int exponent_in(float scale) {
    return imax(kEMin, imin(kEMax, (int)((__float_as_uint(scale) >> 23) & 0xff) - 127));
}

template <bool BF16>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    return BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i])
                : reinterpret_cast<const float *>(p)[i];
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// inv_freq in turns a position, mod 1, in units of 2^-64. 1 / 2 pi is taken in
// two parts, the first of 28 bits, so that its product with a float is exact.
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
    const double hi = (double)inv_freq * (170891318.0 / 1073741824.0);
    const double lo = (double)inv_freq * 8.32702869033044e-10;
    const double two64 = 18446744073709551616.0;
    return (uint64_t)((hi - floor(hi)) * two64) + (uint64_t)((lo - floor(lo)) * two64);
}
__device__ __forceinline__ void sincos_at(int pos, uint64_t f, float &s, float &c) {
    const int32_t turn = (int32_t)(((uint64_t)(uint32_t)pos * f) >> 32);
    sincospif((float)turn * 4.656612873077392578125e-10f, &s, &c);      // 2^-31: half turns
}

// Channel d of the token row at `x`, rotated.
template <bool BF16>
__device__ __forceinline__ float rotated(const AppendArgs &a, const void *x, int64_t row, int d, int pos) {
    const float v = load1<BF16>(x, row + d);
    if (d >= a.rot) return v;
    const int half = a.rot / 2;
    const int j = a.inter ? d >> 1 : (d < half ? d : d - half);
    const bool second = a.inter ? (d & 1) : d >= half;
    const int other = a.inter ? d ^ 1 : (second ? d - half : d + half);
    const float w = load1<BF16>(x, row + other);
    float s, c;
    sincos_at(pos, turns_of(a.inv_freq[j]), s, c);
    return second ? w * s + v * c : v * c - w * s;
}

struct Slot {
    Seq s;
    int b, page, off, count, pos;        // page of the pool, first slot, new tokens, first position
    int64_t t;                           // first token row
};

__device__ __forceinline__ uint8_t e4m3_of(float x) {
    return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float float_of(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// One block a touched page and head: the largest new magnitude, the scale, the
// old codes if it grew, the new codes; keys, then values.
template <bool BF16>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
    __shared__ Slot sl;
    __shared__ float amax_sh[8];
    __shared__ uint32_t bad_sh[4];       // tokens of the page with a non-finite channel
    const int tid = threadIdx.x, D = a.c.D, page = a.c.page, B = a.c.B;
    const int64_t slot = blockIdx.x;
    const int capacity = a.c.W * page;
    if (tid == 0) sl.b = -1;
    if (tid < 4) bad_sh[tid] = 0;
    __syncthreads();
    for (int b = tid; b < B; b += 256) {
        const Seq s = sequence(a.cu, a.n, a.T, a.lens, capacity, b);
        const int64_t first = first_slot(s.t0, b, page);
        const int n = imin(s.n, capacity - s.len);           // what the table has room for
        if (slot == 0 && blockIdx.y == 0) {
            if (!s.ok || n < s.n) atomicCAS(a.status, 0u, (unsigned)kDevBadCache);
            if (a.lens_out) a.lens_out[b] = s.len + n;
        }
        const int i = (int)(slot - first);
        if (slot >= first && i < touched_pages(s.len, n, page)) {
            Slot x;
            x.s = s;
            x.b = b;
            const int at = s.len / page + i;
            x.page = a.c.table[(int64_t)b * a.c.W + at];
            x.off = i == 0 ? s.len % page : 0;
            x.pos = at * page + x.off;
            const int done = x.pos - s.len;
            x.count = imin(page - x.off, n - done);
            x.t = s.t0 + done;
            if (x.page < 0 || x.page >= a.c.P) {
                atomicCAS(a.status, 0u, (unsigned)kDevBadCache);
                x.b = -1;
            }
            sl = x;
        }
    }
    __syncthreads();
    if (sl.b < 0) return;
    const int h = blockIdx.y;
    const Slot x = sl;
    if (h >= a.c.H) {
        // queries: head h - H, rotated and stored
        const int hq = h - a.c.H;
        for (int i = tid; i < x.count * D; i += 256) {
            const int t = i / D, d = i - t * D;
            const float v = rotated<BF16>(a, a.Q, (x.t + t) * a.q_st + (int64_t)hq * D, d, x.pos + t);
            const int64_t o = ((x.t + t) * a.Hq + hq) * D + d;
            if (BF16)
                reinterpret_cast<__nv_bfloat16 *>(a.Q_out)[o] = __float2bfloat16_rn(v);
            else
                reinterpret_cast<float *>(a.Q_out)[o] = v;
        }
        return;
    }
    const int64_t ph = (int64_t)x.page * a.c.H + h;
    for (int i = tid; i < x.count * D; i += 256) {
        const int t = i / D, d = i - t * D;
        const float k = load1<BF16>(a.K, (x.t + t) * a.k_st + (int64_t)h * D + d);
        const float v = load1<BF16>(a.V, (x.t + t) * a.v_st + (int64_t)h * D + d);
        if (!finite(k) || !finite(v)) atomicOr(&bad_sh[t >> 5], 1u << (t & 31));
    }
    for (int kv = 0; kv < 2; ++kv) {
        const void *src = kv ? a.V : a.K;
        const int64_t st = kv ? a.v_st : a.k_st;
        uint8_t *codes = (kv ? a.c.v : a.c.k) + ph * page * D;
        float *scale = (kv ? a.c.vs : a.c.ks) + ph;
        float m = 0.f;
        for (int i = tid; i < x.count * D; i += 256) {
            const int t = i / D, d = i - t * D;
            const float y = fabsf(load1<BF16>(src, (x.t + t) * st + (int64_t)h * D + d));
            if (y < INFINITY) m = fmaxf(m, y);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int was = x.off ? exponent_in(*scale) : kEMin;
        __syncthreads();
        if ((tid & 31) == 0) amax_sh[tid >> 5] = m;
        __syncthreads();
        for (int i = 0; i < 8; ++i) m = fmaxf(m, amax_sh[i]);
        const int e = imax(was, exponent_of(m));
        if (tid == 0) *scale = two_to(e);
        if (e > was)
            for (int i = tid; i < x.off * D; i += 256) codes[i] = e4m3_of(float_of(codes[i]) * two_to(was - e));
        const float inv = two_to(-e);
        for (int i = tid; i < x.count * D; i += 256) {
            const int t = i / D, d = i - t * D;
            const int64_t row = (x.t + t) * st + (int64_t)h * D;
            const bool bad = bad_sh[t >> 5] >> (t & 31) & 1;
            float y;
            if (bad)
                y = kv ? 0.f : NAN;
            else
                y = (kv ? load1<BF16>(src, row + d) : rotated<BF16>(a, src, row, d, x.pos + t)) * inv;
            codes[(x.off + t) * D + d] = e4m3_of(y);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, bool bf16, cudaStream_t st) {
    const dim3 grid((unsigned)slot_bound(a.T, a.c.B, a.c.page), a.c.H + (a.Q ? a.Hq : 0));
    if (bf16)
        append_kernel<true><<<grid, 256, 0, st>>>(a);
    else
        append_kernel<false><<<grid, 256, 0, st>>>(a);
    note_launch();
    return cudaGetLastError();
}

}  // namespace cache
}  // namespace flare
