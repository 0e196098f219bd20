// cache_attn.cu -- attention over the paged 8-bit cache: the CUDA-core kernel,
// the merge of cut items, and the choice of a kernel.
//
// For a query row q of shared head h and the tokens n it sees:
//   S_n = s <q, k_n>,  L = log sum_n exp(S_n),  O = sum_n exp(S_n - L) v_n,
// with k_n, v_n the codes times their page's scales. A running maximum m and
// sum l (fp32) carry the softmax over the tokens in one pass.
#include "cache_device.cuh"

namespace flare {
namespace cache {

// ---- CUDA cores -----------------------------------------------------------------
// R rows a tile, four warps; each warp takes 32 of a tile's 128 tokens, one
// token a lane for S = Q K^T (a lane reads its whole key row, 16 bytes at a
// time; Q is broadcast from shared memory), then four channels a lane for
// O += P V (a warp reads a value row, 4 bytes a lane). Every product is an
// fp32 FMA on exactly converted codes. The reads are as few as they can be
// for one head's rows; the FMAs bound it from some four rows on.
template <int R, bool BF16>
__global__ void __launch_bounds__(128) attn_simt_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int NT = 128, NW = 4;
    __shared__ int64_t scan_sh[NW];
    __shared__ Cursor cur_sh;
    __shared__ __align__(16) float q_sh[R][128];
    __shared__ __align__(16) float p_sh[NW][R][32];
    __shared__ __align__(16) float o_sh[NW][R][128];
    __shared__ float m_sh[NW][R], l_sh[NW][R];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, cta = blockIdx.x;
    const int D = a.c.D;
    const Span sp = find_span<NT>(a, cta, scan_sh, &cur_sh);
    Cursor cur = cur_sh;
    if (tid == 0) write_record(a, sp, cur, cta);
    while (cur.tiles_left > 0) {
        const int k0 = cur.k, k1 = imin(cur.nt, cur.k + cur.tiles_left);
        __syncthreads();
        int limit[R];
#pragma unroll
        for (int r = 0; r < R; ++r) limit[r] = row_place(a, cur.s, cur.b, cur.rt, cur.h, r).limit;
        for (int i = tid; i < R * D; i += NT) {
            const int r = i / D, d = i - r * D;
            const RowPlace p = row_place(a, cur.s, cur.b, cur.rt, cur.h, r);
            q_sh[r][d] = p.valid ? load_q(a, BF16, p.q + d) : 0.f;
        }
        __syncthreads();
        float m[R], l[R];
        float4 o[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
            o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const int seen = visible(cur.s, a.G, a.rows, cur.rt, a.causal);
        for (int k = k0; k < k1; ++k) {
            const int n0 = k * kTile + 32 * w, n = n0 + lane;
            if (n0 >= seen) continue;
            const int page = n < seen ? page_of(a.c, cur.b, n, a.status) : -1;
            const int64_t ph = (int64_t)page * a.c.H + cur.h;
            const int64_t row = (ph * a.c.page + (n & (a.c.page - 1))) * D;
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = 0.f;
            float vs = 0.f, t_scale = 0.f;
            if (page >= 0) {
                t_scale = a.c.ks[ph] * a.sl2;
                vs = a.c.vs[ph];
                for (int d = 0; d < D; d += 16) {
                    const uint4 kq = *reinterpret_cast<const uint4 *>(a.c.k + row + d);
                    const uint32_t kw[4] = {kq.x, kq.y, kq.z, kq.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 x = float2_of(f16x2_of_e4m3x2(kw[c]));
                        const float2 y = float2_of(f16x2_of_e4m3x2_hi(kw[c]));
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float4 q = *reinterpret_cast<const float4 *>(&q_sh[r][d + 4 * c]);
                            s[r] = fmaf(q.x, x.x, s[r]);
                            s[r] = fmaf(q.y, x.y, s[r]);
                            s[r] = fmaf(q.z, y.x, s[r]);
                            s[r] = fmaf(q.w, y.y, s[r]);
                        }
                    }
                }
            }
            // (a lane's value scale goes into its weight for O, not into the sum)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float t = page >= 0 && n < limit[r] ? s[r] * t_scale : -INFINITY;
                float mx = t;
#pragma unroll
                for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mn = fmaxf(m[r], mx);
                const float ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[r] - ref);           // m = -inf: 0
                const float p = exp2f(t - ref);
                m[r] = mn;
                l[r] = l[r] * f + p;
                o[r].x *= f; o[r].y *= f; o[r].z *= f; o[r].w *= f;
                p_sh[w][r][lane] = p * vs;
            }
            __syncwarp();
            const int cnt = imin(32, seen - n0);
            for (int j = 0; j < cnt; ++j) {
                const int64_t vrow = __shfl_sync(0xffffffffu, row, j);
                const int vpage = __shfl_sync(0xffffffffu, page, j);
                if (vpage >= 0 && 4 * lane < D) {
                    const uint32_t c = *reinterpret_cast<const uint32_t *>(a.c.v + vrow + 4 * lane);
                    const float2 x = float2_of(f16x2_of_e4m3x2(c)), y = float2_of(f16x2_of_e4m3x2_hi(c));
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float p = p_sh[w][r][j];
                        o[r].x = fmaf(p, x.x, o[r].x);
                        o[r].y = fmaf(p, x.y, o[r].y);
                        o[r].z = fmaf(p, y.x, o[r].z);
                        o[r].w = fmaf(p, y.y, o[r].w);
                    }
                }
            }
            __syncwarp();
        }
        // the four warps' states of each row become one
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float x = l[r];
#pragma unroll
            for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
            if (lane == 0) {
                m_sh[w][r] = m[r];
                l_sh[w][r] = x;
            }
            if (4 * lane < D) *reinterpret_cast<float4 *>(&o_sh[w][r][4 * lane]) = o[r];
        }
        __syncthreads();
        const bool whole = k0 == 0 && k1 == cur.nt;
        const int64_t slot = (int64_t)cta * 2 + (k0 == 0 ? 1 : 0);
        for (int r = w; r < R; r += NW) {
            const RowPlace p = row_place(a, cur.s, cur.b, cur.rt, cur.h, r);
            if (!p.valid) continue;
            float M = -INFINITY, ls = 0.f;
#pragma unroll
            for (int x = 0; x < NW; ++x) M = fmaxf(M, m_sh[x][r]);
            const float ref = M == -INFINITY ? 0.f : M;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < NW; ++x) {
                const float f = exp2f(m_sh[x][r] - ref);
                ls += l_sh[x][r] * f;
                if (4 * lane < D) {
                    const float4 y = *reinterpret_cast<const float4 *>(&o_sh[x][r][4 * lane]);
                    v.x = fmaf(f, y.x, v.x); v.y = fmaf(f, y.y, v.y);
                    v.z = fmaf(f, y.z, v.z); v.w = fmaf(f, y.w, v.w);
                }
            }
            if (whole) {
                const float inv = ls == 0.f ? 0.f : 1.f / ls;
                if (4 * lane < D)
                    store_o4(a, !BF16 || a.o_f32, p.o + 4 * lane,
                             make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                if (a.L && lane == 0) a.L[p.l] = ls == 0.f ? -INFINITY : (ref + log2f(ls)) * kLn2;
            } else {
                if (4 * lane < D)
                    *reinterpret_cast<float4 *>(&a.part_O[(slot * a.rows + r) * D + 4 * lane]) = v;
                if (lane == 0) a.part_ml[slot * a.rows + r] = make_float2(ref, ls);
            }
        }
        cur.tiles_left -= k1 - k0;
        if (cur.tiles_left > 0) next_item(a, cur);
    }
    tc::pdl_launch_dependents();
}

// ---- merge --------------------------------------------------------------------------
// The item that ends in span blockIdx.x: its pieces lie in spans first ..
// blockIdx.x, the first in slot 1 (it began there) and the rest in slot 0. They are
// added in a fixed order, so results do not vary. A piece without a visible token
// has l = 0. Bound by latency: a few KB a row, in two rounds of loads.
//   ROW: one block a row, its warps share the pieces (few rows of many pieces);
//   else one warp a row (many rows of few pieces).
template <bool ROW>
__global__ void __launch_bounds__(128) attn_merge_kernel(const __grid_constant__ AttnArgs a, const int f32) {
    __shared__ float f_sh[ROW ? kMaxSpans : 1], red[8];
    __shared__ float4 o_sh[ROW ? 3 : 1][32];
    tc::pdl_wait();
    const int4 rec = a.rec[blockIdx.x];
    if (rec.x < 0) return;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int r = ROW ? (int)blockIdx.y : (int)blockIdx.y * 4 + w;
    const int D = a.c.D, first = rec.w, count = (int)blockIdx.x - first + 1;
    if (r >= a.rows) return;
    const Seq s = load_seq(a, rec.x);
    const RowPlace p = row_place(a, s, rec.x, rec.y, rec.z, r);
    if (!p.valid) return;
    const int64_t step = 2 * (int64_t)a.rows, base = (int64_t)first * step + r;
    auto slot = [&](int i) { return base + i * step + (i == 0 ? a.rows : 0); };
    // weights of the pieces; this thread's are i0, i0 + NT, ...
    constexpr int NT = ROW ? 128 : 32;
    const int i0 = ROW ? tid : lane;
    float M = -INFINITY;
    for (int i = i0; i < count; i += NT) {
        const float2 ml = a.part_ml[slot(i)];
        if (!(ml.y == 0.f)) M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    if (ROW) {
        if (lane == 0) red[w] = M;
        __syncthreads();
        M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    }
    const float ref = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float g, int i) {
        if (4 * lane < D) {
            const float4 y = *reinterpret_cast<const float4 *>(&a.part_O[slot(i) * D + 4 * lane]);
            v.x = fmaf(g, y.x, v.x); v.y = fmaf(g, y.y, v.y);
            v.z = fmaf(g, y.z, v.z); v.w = fmaf(g, y.w, v.w);
        }
    };
    auto weight = [&](int i) {
        const float2 ml = a.part_ml[slot(i)];
        const float f = ml.y == 0.f ? 0.f : tc::ex2(ml.x - ref);
        l += f * ml.y;
        return f;
    };
    if (ROW) {
        for (int i = i0; i < count; i += NT) f_sh[i] = weight(i);
        __syncthreads();
#pragma unroll 8
        for (int i = w; i < count; i += 4) add(f_sh[i], i);
    } else {
        for (int b = 0; b < count; b += 32) {
            const float f = b + lane < count ? weight(b + lane) : 0.f;
            const int m = imin(32, count - b);
#pragma unroll 4
            for (int i = 0; i < m; ++i) add(__shfl_sync(0xffffffffu, f, i), b + i);
        }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (ROW) {
        if (lane == 0) red[4 + w] = l;
        if (w > 0) o_sh[w - 1][lane] = v;
        __syncthreads();
        if (w > 0) return;
        l = (red[4] + red[5]) + (red[6] + red[7]);
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const float4 y = o_sh[x][lane];
            v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (4 * lane < D)
        store_o4(a, f32 != 0, p.o + 4 * lane, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    if (a.L && lane == 0) a.L[p.l] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
}

// ---- choice and launch ----------------------------------------------------------------
AttnPlan attn_plan(const Pool &c, int G, bool bf16, int64_t T, bool ragged, int family, int sms) {
    AttnPlan p;
    p.kernel = family == FLARE_KERNEL_SIMT ? AttnKernel::kSimt : AttnKernel::kMma;
    const int64_t per_seq = c.B > 0 ? T * G / c.B : 0;      // rows of a head and sequence on average
    if (p.kernel == AttnKernel::kMma && bf16 && (c.D == 64 || c.D == 128) && per_seq > 32) p.kernel = AttnKernel::kTc;
    p.rows = p.kernel == AttnKernel::kSimt ? 8 : p.kernel == AttnKernel::kTc ? (per_seq > 128 ? 256 : 128)
             : bf16 && per_seq > 16        ? 32
                                           : 16;
    int64_t grid = (int64_t)sms * (p.kernel == AttnKernel::kSimt ? 4 : p.kernel == AttnKernel::kMma ? 2 : 1);
    // Few items of few tokens: clusters of blocks and no merge. Two blocks fit a
    // multiprocessor; a block's share stays under 4096 tokens, beyond which equal spans over
    // all multiprocessors gain more than the second launch costs.
    p.cluster = 1;
    if (p.kernel == AttnKernel::kMma && !ragged && c.B > 0) {
        const int64_t items = (T / c.B * G + p.rows - 1) / p.rows * c.B * c.H;
        for (int s = 8; s > 1 && p.cluster == 1; s /= 2)
            if (items * s <= 2 * sms && (int64_t)c.W * c.page <= 4096 * s) p.cluster = s;
    }
    // no more spans than there can be tiles
    const int64_t tiles = ((T * G + p.rows - 1) / p.rows + c.B) * c.H *
                          (((int64_t)c.W * c.page + kTile - 1) / kTile + 1);
    if (grid > tiles) grid = tiles;
    p.grid = (int)(grid < 1 ? 1 : grid > kMaxSpans ? kMaxSpans : grid);
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    size_t o = up(sizeof(float) * 2 * p.grid * p.rows * c.D);
    p.part_ml = o;
    o += up(sizeof(float2) * 2 * p.grid * p.rows);
    p.rec = o;
    o += up(sizeof(int4) * p.grid);
    p.bytes = o;
    return p;
}

namespace {
template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel k, dim3 grid, dim3 block, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}
}  // namespace

cudaError_t launch_attn(const AttnArgs &a, const AttnPlan &plan, bool bf16, cudaStream_t st) {
    const AttnKernel kernel = plan.kernel;
    cudaError_t e;
    if (kernel == AttnKernel::kSimt) {
        if (bf16)
            attn_simt_kernel<8, true><<<a.grid, 128, 0, st>>>(a);
        else
            attn_simt_kernel<8, false><<<a.grid, 128, 0, st>>>(a);
        note_launch();
        e = cudaGetLastError();
    } else if (kernel == AttnKernel::kTc) {
        e = launch_attn_tc(a, st);
    } else {
        e = launch_attn_mma(a, bf16, plan.cluster, st);
    }
    if (e != cudaSuccess || plan.cluster > 1) return e;
    const int f32 = !bf16 || a.o_f32;
    e = a.rows <= 32 ? launch_pdl(attn_merge_kernel<true>, dim3(a.grid, a.rows), dim3(128), st, a, f32)
                     : launch_pdl(attn_merge_kernel<false>, dim3(a.grid, a.rows / 4), dim3(128), st, a, f32);
    if (e != cudaSuccess) return e;
    note_launch();
    return cudaGetLastError();
}

}  // namespace cache
}  // namespace flare
