// cache_attn_mma.cu -- attention over the paged 8-bit cache for few query rows
// a shared head (one token or a few, times its query heads): split over the
// tokens, bound by reading the cache.
//
// A warp takes 16 tokens at a time (a unit) of one item (sequence, tile of 16 * MT
// rows, head), with a softmax state of its own. Why mma.sync and not tcgen05: a
// 16-row tile meets each code once, and the products of a head's 16 rows are a
// tenth of what the register-operand tensor path does in the time that the codes
// take to arrive; tcgen05 would need them as tiles of 128 rows in shared memory,
// converted and written there first.
//
// Layouts. S = Q K^T and O = P V are m16n8k16 products in fp16 with fp32 sums.
// The order of the channels inside a k-step is free as long as Q and K agree,
// and the order of the output columns is free in P V, so both are chosen to let
// a lane's operands be 16 consecutive codes of a token:
//   K: lane (g, t) = (lane / 4, lane % 4) holds of tokens g and g + 8 the
//      channels 64 j + 16 t .. + 15; k-step (j, s) uses its codes 4 s .. 4 s + 3;
//   V: lane (g, t) holds of tokens 2t, 2t+1, 2t+8, 2t+9 the channels
//      (DP / 8) g .. ; column n of tile j is channel (DP / 8) n + j.
// Each lane copies with cp.async exactly the bytes that it will read, into a
// ring of its warp's own: no barrier, no bank conflict, and the copies of the
// next units are in flight while this one is computed.
//
// Numbers. e4m3 is exact in fp16. A query row is scaled by a power of two so
// that its largest channel lies in [2^14, 2^15): bf16 channels are exact in
// fp16 down to 2^-29 of the largest and below that off by 2^-40 of it; fp32
// ones are split into two fp16 parts (24 bits). A unit's value scale 2^ev goes
// into the exponent of the weights, w = 2^(s + ev - m), and out of their sum:
// O = sum w v8, l = 2^-ev sum w; m is a reference at most 15 below the largest
// s + ev seen, so that w stays under fp16's 65504 and is exact to 2^-11 down to
// 2^-21 of the largest weight. fp32 queries split w into two parts as well.
#include "cache_device.cuh"

namespace flare {
namespace cache {
namespace {

constexpr float kNoMax = -3.0e38f;       // reference before any visible token
constexpr float kHeadroom = 15.f;        // w <= 2^15
constexpr float kFresh = 7.f;            // a new largest score starts at w = 2^7

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on) {
    const int n = on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, bool on) {
    const int n = on ? 8 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool on) {
    const int n = on ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// x - (what pack_f16 kept of it), packed again: the next 11 bits.
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t kept) {
    const float2 k = float2_of(kept);
    return pack_f16(lo - k.x, hi - k.y);
}

__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_size() {
    int r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of block `rank` of the cluster at this block's address `at`.
__device__ __forceinline__ float4 ld_peer4(uint32_t at, int rank) {
    float4 v;
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %4, %5;\n\t"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at), "r"(rank)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t at, int rank) {
    float2 v;
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [p];\n\t}"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(at), "r"(rank)
                 : "memory");
    return v;
}

template <int DP_, int MT_, bool F32_>
struct MmaCfg {
    static constexpr int DP = DP_, MT = MT_;
    static constexpr bool F32 = F32_;
    // two blocks a multiprocessor
    static constexpr int NW = mma_warps(!F32, 16 * MT), NT = 32 * NW;
    static constexpr int ROWS = 16 * MT;
    static constexpr int KJ = DP / 64;                    // 16-byte chunks of a key row a lane holds
    static constexpr int KS = DP / 16;                    // k-steps of S
    static constexpr int NO = DP / 8;                     // column tiles of O
    static constexpr int PARTS = F32 ? 2 : 1;
    static constexpr int VB = DP / 8;                     // bytes of a value row a lane holds
    // one row tile of bf16: Q stays in registers (from shared memory it would be half of the
    // traffic there)
    static constexpr bool QREG = !F32 && MT == 1;
    static constexpr uint32_t UNIT = 32 * (2 * KJ * 16 + 4 * VB) + 256;   // codes, then the scales
    static constexpr uint32_t Q_BYTES = MT * PARTS * KS * 512;
};

// The state of a warp's rows over the tokens it has met, and its queries.
template <class C>
struct State {
    float c[C::MT][2], m[C::MT][2], l[C::MT][2];          // factors of the rows, references, sums
    int lim[C::MT][2], min_lim;                           // tokens that the rows see
    float rest;                                           // what the rounding of the score scale took off
    uint32_t q[C::QREG ? C::KS : 1][4];
    float o[C::MT][C::NO][4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int x = 0; x < C::MT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                m[x][y] = kNoMax;
                l[x][y] = 0.f;
            }
#pragma unroll
        for (int x = 0; x < C::MT; ++x)
#pragma unroll
            for (int j = 0; j < C::NO; ++j)
#pragma unroll
                for (int y = 0; y < 4; ++y) o[x][j][y] = 0.f;
    }
    __device__ __forceinline__ void load_q(uint32_t at, int lane) {
        if (C::QREG)
#pragma unroll
            for (int k = 0; k < C::KS; ++k) {
                const uint4 v = lds16(at + k * 512 + lane * 16);
                constexpr int n = C::QREG ? C::KS : 1;
                q[k % n][0] = v.x; q[k % n][1] = v.y; q[k % n][2] = v.z; q[k % n][3] = v.w;
            }
    }
};

// Copies this lane's bytes of a unit, tokens [n0, n0 + 16) of which those from `end`
// on are zeros, to the ring's slot at st. page < 0: nothing but zeros.
template <class C>
__device__ __forceinline__ void fetch(const AttnArgs &a, int page, int h, int n0, int end, uint32_t st, int lane) {
    constexpr int DP = C::DP, KJ = C::KJ;
    const int g = lane >> 2, t = lane & 3, D = a.c.D;
    const bool ok = page >= 0;
    // where a lane's bytes of a value row lie: the row's together, in an order in which neither
    // the copies of a row nor the lanes of a load meet in a bank
    const uint32_t v_slot = (8 * t + (DP == 128 ? g ^ (2 * t) : g ^ (4 * (t >> 1)))) * C::VB;
    const int64_t ph = (int64_t)(ok ? page : 0) * a.c.H + h;
    const int64_t base = ((ph << a.c.page_log2) + (n0 & (a.c.page - 1))) * D;
    const uint32_t dst = st + lane * 16, vdst = st + 2 * KJ * 512 + v_slot;
    if (ok && n0 + 16 <= end && D == DP) {
        const uint8_t *const ksrc = a.c.k + base + g * DP + 16 * t, *const vsrc = a.c.v + base + 2 * t * DP + C::VB * g;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < KJ; ++j) cp16(dst + (r * KJ + j) * 512, ksrc + 8 * r * DP + 64 * j, true);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint8_t *src = vsrc + ((r & 1) + 8 * (r >> 1)) * DP;
            if (DP == 128)
                cp16(vdst + r * 32 * C::VB, src, true);
            else
                cp8(vdst + r * 32 * C::VB, src, true);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                const int row = g + 8 * r, ch = 64 * j + 16 * t;
                const bool on = ok && n0 + row < end && ch < D;
                cp16(dst + (r * KJ + j) * 512, a.c.k + (on ? base + row * D + ch : 0), on);
            }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + 8 * (r >> 1), ch = C::VB * g;
            const bool on = ok && n0 + row < end && ch < D;
            const uint8_t *src = a.c.v + (on ? base + row * D + ch : 0);
            if (DP == 128)
                cp16(vdst + r * 32 * C::VB, src, on);
            else
                cp8(vdst + r * 32 * C::VB, src, on);
        }
    }
    const uint32_t sdst = st + C::UNIT - 256 + lane * 8;
    cp4(sdst, a.c.ks + ph, ok);
    cp4(sdst + 4, a.c.vs + ph, ok);
}

// S = Q K^T, the weights and O += w V of the unit in slot st, tokens n0 .. n0 + 15;
// those from `end` on are hidden. q_at: the queries, where they are not in registers.
template <class C>
__device__ __forceinline__ void unit(State<C> &z, uint32_t st, uint32_t q_at, int n0, int end, int lane) {
    constexpr int DP = C::DP, MT = C::MT, KJ = C::KJ, KS = C::KS, NO = C::NO;
    constexpr bool F32 = C::F32, QREG = C::QREG;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t v_slot = (8 * t + (DP == 128 ? g ^ (2 * t) : g ^ (4 * (t >> 1)))) * C::VB;
    auto &c = z.c;
    auto &m = z.m;
    auto &l = z.l;
    auto &o = z.o;
    auto &lim = z.lim;
    float s[MT][2][4];
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x][n][y] = 0.f;
    // float32: the two parts apart and 64 channels at a time, since the tensor cores cut a sum
    // off where they do not round it
    float hi[MT][2][4], lo[MT][2][4];
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int y = 0; y < 4; ++y) hi[x][n][y] = lo[x][n][y] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
        const uint4 ka = lds16(st + j * 512 + lane * 16), kb = lds16(st + (KJ + j) * 512 + lane * 16);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t a0 = f16x2_of_e4m3x2(wa[q]), a1 = f16x2_of_e4m3x2_hi(wa[q]);
            const uint32_t b0 = f16x2_of_e4m3x2(wb[q]), b1 = f16x2_of_e4m3x2_hi(wb[q]);
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
                for (int part = C::PARTS - 1; part >= 0; --part) {
                    uint32_t f[4];
                    if (QREG) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) f[y] = z.q[(j * 4 + q) % (QREG ? KS : 1)][y];
                    } else {
                        const uint4 v = lds16(q_at + ((x * C::PARTS + part) * KS + j * 4 + q) * 512 + lane * 16);
                        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
                    }
                    float (&to)[2][4] = !F32 ? s[x] : part ? lo[x] : hi[x];
                    mma16816(to[0], f, a0, a1);
                    mma16816(to[1], f, b0, b1);
                }
        }
        if (F32)
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        s[x][n][y] += j + 1 < KJ ? hi[x][n][y] : hi[x][n][y] + lo[x][n][y];
                        hi[x][n][y] = 0.f;
                    }
    }
    const uint2 sc = lds8(st + C::UNIT - 256 + lane * 8);
    const float ks = __uint_as_float(sc.x), vs = __uint_as_float(sc.y);
    const float ev = (float)((int)(sc.y >> 23) - 127);
    const float inv_vs = __int_as_float((254 - (int)(sc.y >> 23)) << 23);
    const bool whole = vs != 0.f && n0 + 16 <= z.min_lim;
    uint32_t pf[MT][4], pr[MT][4];
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const float cc = c[x][y] * ks;
            const float v[4] = {s[x][0][2 * y], s[x][0][2 * y + 1], s[x][1][2 * y], s[x][1][2 * y + 1]};
            unsigned hidden = 0;
            if (!whole)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = n0 + 2 * t + (e & 1) + 8 * (e >> 1);
                    if (vs == 0.f || n >= lim[x][y] || n >= end) hidden |= 1u << e;
                }
            // Exponents of the weights against reference `ref`. float32: ref is a whole number, so
            // that ev - ref is exact and what is rounded is small where the weight is large, and
            // the rounding of the score scale is made up for (either would put scores of 40 off by
            // 2e-6). bf16: ref is such that the largest weight met so far is a power of two, which
            // fp16 holds without a rounding.
            float u[4];
            auto exponents = [&](float ref) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    u[e] = fmaf(v[e], cc, ev - ref);
                    if (F32) u[e] = fmaf(v[e] * cc, z.rest, u[e]);
                    if (hidden >> e & 1) u[e] = -INFINITY;
                }
                return fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3]));
            };
            if (__any_sync(0xffffffffu, exponents(m[x][y]) > kHeadroom)) {
                float best = exponents(0.f);
                best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
                best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
                if (best > m[x][y] + kHeadroom) {
                    const float top = F32 ? rintf(best - kFresh) : best - kFresh, f = tc::ex2(m[x][y] - top);
                    m[x][y] = top;
                    l[x][y] *= f;
#pragma unroll
                    for (int j = 0; j < NO; ++j) {
                        o[x][j][2 * y] *= f;
                        o[x][j][2 * y + 1] *= f;
                    }
                }
                exponents(m[x][y]);
            }
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = tc::ex2(u[e]);
            l[x][y] = fmaf((p[0] + p[1]) + (p[2] + p[3]), inv_vs, l[x][y]);
            pf[x][y] = pack_f16(p[0], p[1]);
            pf[x][2 + y] = pack_f16(p[2], p[3]);
            if (F32) {
                pr[x][y] = pack_rest(p[0], p[1], pf[x][y]);
                pr[x][2 + y] = pack_rest(p[2], p[3], pf[x][2 + y]);
            }
        }
    // O += P V
    uint32_t vr[4][C::VB / 4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const uint32_t at = st + 2 * KJ * 512 + y * 32 * C::VB + v_slot;
        if (DP == 128) {
            const uint4 v = lds16(at);
            vr[y][0] = v.x; vr[y][1] = v.y; vr[y][C::VB / 4 - 2] = v.z; vr[y][C::VB / 4 - 1] = v.w;
        } else {
            const uint2 v = lds8(at);
            vr[y][0] = v.x; vr[y][1] = v.y;
        }
    }
#pragma unroll
    for (int q = 0; q < C::VB / 4; ++q) {
        const uint32_t r[4] = {vr[0][q], vr[1][q], vr[2][q], vr[3][q]};
        const uint32_t lo01 = __byte_perm(r[0], r[1], 0x5140), hi01 = __byte_perm(r[0], r[1], 0x7362);
        const uint32_t lo23 = __byte_perm(r[2], r[3], 0x5140), hi23 = __byte_perm(r[2], r[3], 0x7362);
        const uint32_t b0[4] = {f16x2_of_e4m3x2(lo01), f16x2_of_e4m3x2_hi(lo01), f16x2_of_e4m3x2(hi01),
                                f16x2_of_e4m3x2_hi(hi01)};
        const uint32_t b1[4] = {f16x2_of_e4m3x2(lo23), f16x2_of_e4m3x2_hi(lo23), f16x2_of_e4m3x2(hi23),
                                f16x2_of_e4m3x2_hi(hi23)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int x = 0; x < MT; ++x) {
                if (F32) {
                    // The tensor cores cut a sum off where they do not round it: into o that would
                    // take a bit off what a large weight left there with every unit that follows,
                    // so the unit's share is added with a rounding.
                    float v[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816(v, pr[x], b0[j], b1[j]);
                    mma16816(v, pf[x], b0[j], b1[j]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[x][4 * q + j][y] += v[y];
                } else {
                    mma16816(o[x][4 * q + j], pf[x], b0[j], b1[j]);
                }
            }
    }
}

// A warp's units of an item: first, first + stride, ... (mine of them, 16 tokens each,
// hidden from token `end` on), through the warp's own ring of STAGES slots at `ring`.
template <class C, int STAGES>
struct Reader {
    const AttnArgs &a;
    const uint32_t ring;
    const int lane;
    const int32_t *table;
    int h, first, stride, mine, end;
    int pg, pg_next;                     // lane i: the page of unit 32 n + i, and of 32 (n + 1) + i
    __device__ __forceinline__ Reader(const AttnArgs &args, uint32_t at, int ln) : a(args), ring(at), lane(ln), mine(0) {}
    __device__ __forceinline__ int page_at(int i) const {
        if (i >= mine) return -1;
        const int p = table[((first + i * stride) * 16) >> a.c.page_log2];
        if (p < 0 || p >= a.c.P) {
            flag_bad(a.status);
            return -1;
        }
        return p;
    }
    __device__ __forceinline__ uint32_t slot(int i) const { return ring + (uint32_t)(i % STAGES) * C::UNIT; }
    __device__ __forceinline__ void issue(int i) {
        if (i < mine) {
            if ((i & 31) == 0) {
                if (i > 0) pg = pg_next;
                pg_next = page_at(i + 32 + lane);
            }
            fetch<C>(a, __shfl_sync(0xffffffffu, pg, i & 31), h, (first + i * stride) * 16, end, slot(i), lane);
        }
        tc::cp_async_commit();
    }
    // The copies of all but the last slot set off. That one is free until read().
    __device__ __forceinline__ void begin(int b, int head, int first_unit, int step, int count, int limit) {
        table = a.c.table + (int64_t)b * a.c.W;
        h = head;
        first = first_unit;
        stride = step;
        mine = count;
        end = limit;
        pg = page_at(lane);
        pg_next = -1;
#pragma unroll 1
        for (int i = 0; i < STAGES - 1; ++i) issue(i);
    }
    __device__ __forceinline__ void read(State<C> &z, uint32_t q_at) {
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            cp_wait<STAGES - 2>();
            unit<C>(z, slot(i), q_at, (first + i * stride) * 16, end, lane);
            issue(i + STAGES - 1);
        }
        cp_wait<0>();
    }
};

// The warp's rows: their queries as fragments at q_at (and from there in registers, where
// they stay there), their factors and limits. A lane holds of rows g and g + 8 of a tile
// the channels that its keys hold: 64 j + 16 t .. + 15.
template <class C>
__device__ __forceinline__ void load_rows(const AttnArgs &a, const Cursor &cur, int rows, int end, State<C> &z, uint32_t q_at,
                                          int lane) {
    const int g = lane >> 2, t = lane & 3, D = a.c.D;
    z.min_lim = end;
    z.rest = a.sl2_rest;
#pragma unroll 1
    for (int rr = 0; rr < 2 * C::MT; ++rr) {
        float x[C::KJ][2][8];
#pragma unroll
        for (int j = 0; j < C::KJ; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[j][0][i] = x[j][1][i] = 0.f;
        float f = 0.f;
        int lim = end;
        if (8 * rr < rows) {
            const RowPlace p = row_place(a, cur.s, cur.b, cur.rt, cur.h, 8 * rr + g);
            if (p.valid) lim = p.limit;
#pragma unroll
            for (int j = 0; j < C::KJ; ++j)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int ch = 64 * j + 16 * t + 8 * y;
                    if (p.valid && ch < D) load_q8(a, !C::F32, p.q + ch, x[j][y]);
                }
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < C::KJ; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = max(top, max(__float_as_uint(x[j][0][i]) & 0x7fffffffu, __float_as_uint(x[j][1][i]) & 0x7fffffffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = imax((int)(top >> 23) - 127, -100);
        const float inv = __int_as_float((14 - e + 127) << 23);      // e <= 127: a normal number
        f = top >= 0x7f800000u ? NAN : __int_as_float((e - 14 + 127) << 23) * a.sl2;
#pragma unroll
        for (int n = 0; n < 2 * C::MT; ++n)
            if (n == rr) {
                z.c[n >> 1][n & 1] = f;
                z.lim[n >> 1][n & 1] = lim;
            }
        z.min_lim = imin(z.min_lim, lim);
        const uint32_t at = q_at + (rr >> 1) * C::PARTS * C::KS * 512 + lane * 16 + (rr & 1) * 4;
#pragma unroll
        for (int j = 0; j < C::KJ; ++j)
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float y0 = x[j][i >> 3][i & 7] * inv, y1 = x[j][i >> 3][(i & 7) + 1] * inv;
                const uint32_t q = pack_f16(y0, y1), to = at + (j * 4 + (i >> 2)) * 512 + (i >> 1 & 1) * 8;
                sts4(to, q);
                if (C::F32) sts4(to + C::KS * 512, pack_rest(y0, y1, q));
            }
    }
    z.min_lim = __reduce_min_sync(0xffffffffu, z.min_lim);
    __syncwarp();
    z.load_q(q_at, lane);
    z.clear();
    __syncwarp();                                                // q_at may be written again
}

// Sum of a row over the four lanes that hold it.
__device__ __forceinline__ float over_row(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// ---- spans of warps ---------------------------------------------------------------
// Every warp has an equal span of the call's tiles (of 32 tokens, and kItemTiles for
// beginning an item) for itself: no barrier, and no joining but at the spans' ends. A
// piece's first codes are on their way before the piece before it is written. Two blocks
// of six warps a multiprocessor, three units of each warp on their way (100 KB).
// Against spans of whole blocks, whose warps took an item's units in turn and joined at
// its end, with 8 heads of 128 and 4 queries each, in a replayed graph: 64 sequences of 0
// to 8,000 tokens 195 -> 101 us, 512 of 0 to 1,000 333 -> 116 (half of either by
// kItemTiles: with 0 instead of 4 135 and 265), 32 of 0 to 16,000 117 -> 100 (553 MB in
// all, 5.5 TB/s); 1,000,003 tokens of one sequence 297 -> 306 (6.7 TB/s: a merge of 228
// pieces a head instead of 38; block spans for that case alone, their units in turn, were
// no faster).
template <class C>
struct SpanCfg {
    static constexpr int STAGES = C::DP == 128 ? 4 : C::NW == 6 ? 7 : 8;
    static constexpr uint32_t RING = STAGES * C::UNIT;
    static constexpr uint32_t WARP = RING + (C::QREG ? 0 : C::Q_BYTES);       // registers: the last slot serves
    static constexpr uint32_t BYTES = C::NW * WARP;
    static_assert(!C::QREG || C::Q_BYTES <= C::UNIT, "a slot is too small for the queries");
    static_assert(8 * (C::DP + 4) * 4 <= C::UNIT, "a slot is too small for eight rows of the output");
    static_assert(2 * (BYTES + 1024 + 512) <= 233472, "shared memory of two CTAs exceeded");
};
template <class C>
__global__ void __launch_bounds__(C::NT, 2) attn_mma_span_kernel(const __grid_constant__ AttnArgs a) {
    using S = SpanCfg<C>;
    constexpr int NW = C::NW, DP = C::DP;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int D = a.c.D;
    const uint32_t ring = tc::smem_u32(smem) + w * S::WARP, spare = ring + (S::STAGES - 1) * C::UNIT;
    const uint32_t q_at = C::QREG ? spare : ring + S::RING;
    float *const out = reinterpret_cast<float *>(smem + w * S::WARP + (S::STAGES - 1) * C::UNIT);
    Cursor cur;
    const Span sp = find_spans<C::NT, NW, kWarpTile>(a, cur);
    const int part = sp.part;
    if (lane == 0 && part < a.grid) write_record(a, sp, cur, part);
    Reader<C, S::STAGES> in(a, ring, lane);
    State<C> z;
    int k0, k1;
    auto begin = [&]() {
        k0 = cur.k;
        k1 = imin(cur.nt, cur.k + cur.tiles_left);
        const int end = imin(visible(cur.s, a.G, a.rows, cur.rt, a.causal), k1 * kWarpTile);
        const int first = k0 * (kWarpTile / 16);
        in.begin(cur.b, cur.h, first, 1, imax(0, (end + 15) / 16 - first), end);
    };
    if (cur.tiles_left > 0) begin();
    while (cur.tiles_left > 0) {
        const int rows = imin(C::ROWS, cur.s.n * a.G - cur.rt * C::ROWS);      // of the tile that are someone's
        if (in.mine > 0) {
            load_rows<C>(a, cur, rows, in.end, z, q_at, lane);
            in.read(z, q_at);
        } else {
            z.clear();
        }
        // ---- the piece is done: the next one's codes first -------------------------------
        const Cursor was = cur;
        const bool final = k0 == 0 && k1 == cur.nt;
        const int64_t slot = (int64_t)part * 2 + (k0 == 0 ? 1 : 0);
        cur.tiles_left -= k1 - k0;
        __syncwarp();
        if (cur.tiles_left > 0) {
            next_item<kWarpTile>(a, cur);
            begin();
        }
#pragma unroll
        for (int x = 0; x < C::MT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r0 = 16 * x + 8 * y;
                if (r0 >= rows) break;
                // rows r0 .. r0 + 7 through the slot that nothing is on its way to, in order
                const float l = over_row(z.l[x][y]), m = z.m[x][y];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < C::NO; j += 4)
                        *reinterpret_cast<float4 *>(&out[g * (DP + 4) + C::VB * (2 * t + e) + j]) =
                            make_float4(z.o[x][j][2 * y + e], z.o[x][j + 1][2 * y + e], z.o[x][j + 2][2 * y + e],
                                        z.o[x][j + 3][2 * y + e]);
                __syncwarp();
                constexpr int LR = DP / 4, RW = 32 / LR;          // lanes a row, rows at a time
                const int d = 4 * (lane % LR);
#pragma unroll 1
                for (int i = 0; i < imin(8, rows - r0); i += RW) {
                    const int r = i + lane / LR;
                    const float lr = __shfl_sync(0xffffffffu, l, 4 * r), mr = __shfl_sync(0xffffffffu, m, 4 * r);
                    if (r0 + r >= rows || d >= D) continue;
                    const float4 v = *reinterpret_cast<const float4 *>(&out[r * (DP + 4) + d]);
                    if (final) {
                        const RowPlace p = row_place(a, was.s, was.b, was.rt, was.h, r0 + r);
                        const float inv = lr == 0.f ? 0.f : 1.f / lr;
                        store_o4(a, C::F32 || a.o_f32, p.o + d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                        if (a.L && d == 0) a.L[p.l] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
                    } else {
                        *reinterpret_cast<float4 *>(&a.part_O[(slot * a.rows + r0 + r) * D + d]) = v;
                        if (d == 0) a.part_ml[slot * a.rows + r0 + r] = make_float2(mr, lr);
                    }
                }
                __syncwarp();
            }
    }
    tc::pdl_launch_dependents();
}

// ---- clusters -------------------------------------------------------------------------
// A cluster of blocks takes one item, each warp of them an equal share of its units, and
// joins their states through shared memory and distributed shared memory: one launch and
// no workspace, for calls so small that a second launch would cost as much as the
// attention. One token of 4 queries a head, 8 heads of 128, 1,500 tokens: 8.1 us; 3 tokens
// of 5 queries, 6 sequences of 2 to 9,000, 4 heads of 64: 18.5 (the longest sequence's 563
// units are 12 rounds of its 48 warps); float32, 500 to 7,000 tokens, 4 heads of 64: 15.1.
// The states of a block's warps become one: sink(r, d, M, l, v) gets channels d .. d + 3 of
// row r, with reference M and sum l. `at`: shared memory (JOIN bytes) that the warps may
// have used until now.
template <class C>
struct JoinCfg {
    static constexpr uint32_t OS = C::DP + 8;             // padded row
    static constexpr uint32_t ML = C::NW * C::ROWS * OS;  // m, l of each warp and row behind them
    static constexpr uint32_t BYTES = (ML + 2 * C::NW * C::ROWS) * 4;
};
template <class C, class Sink>
__device__ __forceinline__ void join_warps(const State<C> &z, int rows, int D, float *at, Sink sink) {
    using J = JoinCfg<C>;
    constexpr int NW = C::NW, ROWS = C::ROWS, DP = C::DP;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
    float *const m_sh = at + J::ML, *const l_sh = m_sh + NW * ROWS;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < C::MT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const float l = over_row(z.l[x][y]);
            const int r = 16 * x + 8 * y + g;
            if (r < rows) {
                if (t == 0) {
                    m_sh[w * ROWS + r] = z.m[x][y];
                    l_sh[w * ROWS + r] = l;
                }
#pragma unroll
                for (int j = 0; j < C::NO; ++j)
                    *reinterpret_cast<float2 *>(&at[(w * ROWS + r) * J::OS + 8 * j + 2 * t]) =
                        make_float2(z.o[x][j][2 * y], z.o[x][j][2 * y + 1]);
            }
        }
    __syncthreads();
    for (int i = tid; i < rows * (DP / 4); i += C::NT) {
        const int r = i / (DP / 4), d = (i % (DP / 4)) * 4;
        if (d >= D) continue;
        float M = kNoMax, ls = 0.f;
#pragma unroll
        for (int x = 0; x < NW; ++x) M = fmaxf(M, m_sh[x * ROWS + r]);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        const int n = d / C::VB, j = d % C::VB;           // channel d = VB n + j
#pragma unroll
        for (int x = 0; x < NW; ++x) {
            const float f = tc::ex2(m_sh[x * ROWS + r] - M);
            ls = fmaf(f, l_sh[x * ROWS + r], ls);
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = fmaf(f, at[(x * ROWS + r) * J::OS + 8 * (j + y) + n], v[y]);
        }
        sink(r, d, M, ls, make_float4(v[0], v[1], v[2], v[3]));
    }
}

template <class C>
struct ClusterCfg {
    static constexpr int STAGES = C::DP == 128 ? (C::NW == 6 ? 3 : 4) : 7;
    static constexpr uint32_t RING = C::NW * STAGES * C::UNIT;
    static constexpr uint32_t JOIN = (JoinCfg<C>::BYTES + 15) / 16 * 16;
    static constexpr uint32_t Q_OFF = RING > JOIN ? RING : JOIN;
    static constexpr uint32_t END = Q_OFF + (C::QREG ? 0 : C::NW * C::Q_BYTES);
    // a cluster's exchange: this block's O, m and l of each row, where queries were
    static constexpr uint32_t EX = C::ROWS * (C::DP * 4 + 8);
    static constexpr uint32_t EX_OFF = Q_OFF;
    static constexpr uint32_t BYTES = C::QREG ? EX_OFF + EX : END;
    static_assert(C::QREG || EX <= C::NW * C::Q_BYTES, "the exchange is larger than the queries");
    static_assert(2 * (BYTES + 1024 + 512) <= 233472, "shared memory of two CTAs exceeded");
};
template <class C>
__global__ void __launch_bounds__(C::NT, 2) attn_mma_cluster_kernel(const __grid_constant__ AttnArgs a) {
    using S = ClusterCfg<C>;
    constexpr int NW = C::NW, NT = C::NT, ROWS = C::ROWS, DP = C::DP;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int D = a.c.D, shares = cluster_size(), share = cluster_rank();
    const uint32_t ring = tc::smem_u32(smem) + w * S::STAGES * C::UNIT;
    const uint32_t q_at = C::QREG ? ring + (S::STAGES - 1) * C::UNIT : tc::smem_u32(smem) + S::Q_OFF + w * C::Q_BYTES;
    float *const ex_o = reinterpret_cast<float *>(smem + S::EX_OFF);
    float2 *const ex_ml = reinterpret_cast<float2 *>(ex_o + ROWS * DP);

    Cursor cur;
    const int item = (int)blockIdx.x / shares, tiles = row_tiles({0, a.n, 0, true}, a.G, a.rows);
    cur.h = item % a.c.H;
    cur.rt = item / a.c.H % tiles;
    cur.b = item / a.c.H / tiles;
    cur.s = load_seq(a, cur.b);
    if (!cur.s.ok && tid == 0) flag_bad(a.status);
    const int seen = visible(cur.s, a.G, a.rows, cur.rt, a.causal), all = (seen + 15) / 16;
    const int u0 = (int)((int64_t)all * share / shares), u1 = (int)((int64_t)all * (share + 1) / shares);
    const int units = u1 - u0, rows = imin(ROWS, cur.s.n * a.G - cur.rt * ROWS);
    Reader<C, S::STAGES> in(a, ring, lane);
    in.begin(cur.b, cur.h, u0 + w, NW, units > w ? (units - w + NW - 1) / NW : 0, imin(seen, 16 * u1));
    State<C> z;
    load_rows<C>(a, cur, rows, in.end, z, q_at, lane);
    in.read(z, q_at);
    join_warps(z, rows, D, reinterpret_cast<float *>(smem), [&](int r, int d, float M, float l, float4 v) {
        *reinterpret_cast<float4 *>(&ex_o[r * DP + d]) = v;
        if (d == 0) ex_ml[r] = make_float2(M, l);
    });
    cluster_sync();
    // the blocks share the rows' channels out among them
    for (int i = tid * shares + share; i < rows * (DP / 4); i += NT * shares) {
        const int r = i / (DP / 4), d = (i % (DP / 4)) * 4;
        if (d >= D) continue;
        const RowPlace p = row_place(a, cur.s, cur.b, cur.rt, cur.h, r);
        const uint32_t ml = tc::smem_u32(&ex_ml[r]), at = tc::smem_u32(&ex_o[r * DP + d]);
        float M = kNoMax, ls = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = 0; x < shares; ++x) M = fmaxf(M, ld_peer2(ml, x).x);
        for (int x = 0; x < shares; ++x) {
            const float2 y = ld_peer2(ml, x);
            const float4 o4 = ld_peer4(at, x);
            const float f = y.y == 0.f ? 0.f : tc::ex2(y.x - M);
            ls = fmaf(f, y.y, ls);
            v.x = fmaf(f, o4.x, v.x); v.y = fmaf(f, o4.y, v.y);
            v.z = fmaf(f, o4.z, v.z); v.w = fmaf(f, o4.w, v.w);
        }
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        store_o4(a, C::F32 || a.o_f32, p.o + d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        if (a.L && d == 0) a.L[p.l] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * kLn2;
    }
    cluster_sync();                                  // no block leaves while another reads it
}

template <class K>
cudaError_t launch_as(K k, SharedMemoryLimit &limit, const AttnArgs &a, unsigned grid, int threads, uint32_t bytes, int cluster,
                      cudaStream_t st) {
    cudaError_t e = limit.raise((const void *)k, (int)bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, k, a);
    note_launch();
    return e == cudaSuccess ? cudaGetLastError() : e;
}
template <int DP, int MT, bool F32>
cudaError_t launch_mma(const AttnArgs &a, const AttnPlan &plan, cudaStream_t st) {
    using C = MmaCfg<DP, MT, F32>;
    static SharedMemoryLimit spans, clusters;
    if (plan.cluster > 1) {
        const int64_t items = (int64_t)a.c.B * a.c.H * row_tiles({0, a.n, 0, true}, a.G, a.rows);
        return launch_as(attn_mma_cluster_kernel<C>, clusters, a, (unsigned)items * plan.cluster, C::NT, ClusterCfg<C>::BYTES,
                         plan.cluster, st);
    }
    return launch_as(attn_mma_span_kernel<C>, spans, a, (unsigned)plan.blocks, C::NT, SpanCfg<C>::BYTES, 1, st);
}

}  // namespace

cudaError_t launch_attn_mma(const AttnArgs &a, const AttnPlan &plan, bool bf16, cudaStream_t st) {
    const bool wide = a.c.D > 64, two = a.rows == 32;
    if (bf16) {
        if (wide) return two ? launch_mma<128, 2, false>(a, plan, st) : launch_mma<128, 1, false>(a, plan, st);
        return two ? launch_mma<64, 2, false>(a, plan, st) : launch_mma<64, 1, false>(a, plan, st);
    }
    return wide ? launch_mma<128, 1, true>(a, plan, st) : launch_mma<64, 1, true>(a, plan, st);
}

}  // namespace cache
}  // namespace flare
