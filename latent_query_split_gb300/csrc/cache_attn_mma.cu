// cache_attn_mma.cu -- attention over the paged 8-bit cache for few query rows
// a shared head (one token or a few, times its query heads): split over the
// tokens, bound by reading the cache.
//
// Per (sequence, head, tile of 16 * MT rows) the CTA's warps take units of 16
// tokens in turn, each with a softmax state of its own, joined at the end of
// the piece. Why mma.sync and not tcgen05: a 16-row tile meets each code once,
// and the products of a head's 16 rows are a tenth of what the register-operand
// tensor path does in the time that the codes take to arrive; tcgen05 would
// need them as tiles of 128 rows in shared memory, converted and written there
// first.
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

template <int DP, int MT, bool F32, bool CL>
struct MmaCfg {
    // two blocks a multiprocessor: one's loads run while the other joins its warps, writes and
    // begins its next piece
    static constexpr int NW = MT == 1 && !F32 ? 6 : 4, NT = 32 * NW;
    static constexpr int ROWS = 16 * MT;
    static constexpr int KJ = DP / 64;                    // 16-byte chunks of a key row a lane holds
    static constexpr int KS = DP / 16;                    // k-steps of S
    static constexpr int NO = DP / 8;                     // column tiles of O
    static constexpr int PARTS = F32 ? 2 : 1;
    static constexpr int VB = DP / 8;                     // bytes of a value row a lane holds
    static constexpr uint32_t UNIT = 32 * (2 * KJ * 16 + 4 * VB) + 256;   // codes, then the scales
    static constexpr int STAGES = (DP == 128 ? (NW == 6 ? 4 : 5) : 8) - (CL ? 1 : 0);
    static constexpr uint32_t RING = NW * STAGES * UNIT;
    static constexpr uint32_t OS = DP + 8;                // padded row of the joining buffer
    static constexpr uint32_t JOIN = NW * ROWS * OS * 4;
    static constexpr uint32_t Q_OFF = RING > JOIN ? RING : JOIN;
    static constexpr uint32_t Q_BYTES = MT * PARTS * KS * 512;
    static constexpr uint32_t ML_OFF = Q_OFF + Q_BYTES;   // m, l of each warp and row; row factors
    // a cluster's exchange: this block's O, m and l of each row
    static constexpr uint32_t EX_OFF = (ML_OFF + 2 * NW * ROWS * 4 + ROWS * 4 + 15) / 16 * 16;
    static constexpr uint32_t BYTES = EX_OFF + (CL ? ROWS * (DP * 4 + 8) : 0);
    static_assert(2 * (BYTES + 1024 + 512) <= 233472, "shared memory of two CTAs exceeded");
};

// CL: a cluster of blocks takes one item, each block an equal share of its tokens,
// and joins them through distributed shared memory: one launch and no workspace,
// for calls so small that a second launch would cost as much as the attention.
template <int DP, int MT, bool F32, bool CL>
__global__ void __launch_bounds__(MmaCfg<DP, MT, F32, CL>::NT, 2) attn_mma_kernel(const __grid_constant__ AttnArgs a) {
    using C = MmaCfg<DP, MT, F32, CL>;
    constexpr int NW = C::NW, NT = C::NT, ROWS = C::ROWS, KJ = C::KJ, KS = C::KS, NO = C::NO, STAGES = C::STAGES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan_sh[NW];
    __shared__ Cursor cur_sh;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, cta = blockIdx.x;
    const int g = lane >> 2, t = lane & 3;
    const int D = a.c.D, page_log2 = a.c.page_log2, H = a.c.H;
    const uint32_t sbase = tc::smem_u32(smem);
    const int k_off = g * DP + 16 * t, v_off = 2 * t * DP + C::VB * g;      // this lane's first bytes (D = DP)
    // where a lane's bytes of a value row lie: the row's together, in an order in which neither
    // the copies of a row nor the lanes of a load meet in a bank
    const uint32_t v_slot = (8 * t + (DP == 128 ? g ^ (2 * t) : g ^ (4 * (t >> 1)))) * C::VB;
    const uint32_t ring = sbase + (uint32_t)w * STAGES * C::UNIT;
    float *const join = reinterpret_cast<float *>(smem);
    float *const m_sh = reinterpret_cast<float *>(smem + C::ML_OFF), *const l_sh = m_sh + NW * ROWS;
    float *const factor = l_sh + NW * ROWS;
    float *const ex_o = reinterpret_cast<float *>(smem + C::EX_OFF);
    float2 *const ex_ml = reinterpret_cast<float2 *>(ex_o + ROWS * DP);

    Cursor cur;
    int share = 0, shares = 1;
    if (CL) {
        shares = cluster_size();
        share = cluster_rank();
        const int item = cta / shares, m = row_tiles({0, a.n, 0, true}, a.G, a.rows);
        cur.h = item % a.c.H;
        cur.rt = item / a.c.H % m;
        cur.b = item / a.c.H / m;
        cur.s = load_seq(a, cur.b);
        if (!cur.s.ok && tid == 0) flag_bad(a.status);
        cur.k = 0;
        cur.nt = cur.tiles_left = 1;
    } else {
        const Span sp = find_span<NT>(a, cta, scan_sh, &cur_sh);
        cur = cur_sh;
        if (tid == 0) write_record(a, sp, cur, cta);
    }

    while (cur.tiles_left > 0) {
        const int k0 = cur.k, k1 = imin(cur.nt, cur.k + cur.tiles_left);
        const int seen = visible(cur.s, a.G, a.rows, cur.rt, a.causal);
        // tokens up to `end` and units from u0 on are this block's
        int end, u0;
        if (CL) {
            const int all = (seen + 15) / 16;
            u0 = (int)((int64_t)all * share / shares);
            end = imin(seen, 16 * (int)((int64_t)all * (share + 1) / shares));
        } else {
            end = imin(seen, k1 * kTile);
            u0 = k0 * (kTile / 16);
        }
        const int units = imax(0, (end + 15) / 16 - u0);
        const int mine = units > w ? (units - w + NW - 1) / NW : 0;   // this warp's units: u0 + w + i NW
        const int32_t *const row_table = a.c.table + (int64_t)cur.b * a.c.W;
        // ---- pages: lane i holds that of unit base + i of this warp -----------------
        auto page_at = [&](int i) -> int {
            if (i >= mine) return -1;
            const int p = row_table[((u0 + w + i * NW) * 16) >> page_log2];
            if (p < 0 || p >= a.c.P) {
                flag_bad(a.status);
                return -1;
            }
            return p;
        };
        int pg = page_at(lane), pg_next = -1;
        auto issue = [&](int i) {
            if (i < mine) {
                if ((i & 31) == 0) {
                    if (i > 0) pg = pg_next;
                    pg_next = page_at(i + 32 + lane);
                }
                const int page = __shfl_sync(0xffffffffu, pg, i & 31);
                const int n0 = (u0 + w + i * NW) * 16;
                const bool ok = page >= 0;
                const int64_t ph = (int64_t)(ok ? page : 0) * H + cur.h;
                const int64_t base = ((ph << page_log2) + (n0 & (a.c.page - 1))) * D;
                const uint32_t st = ring + (uint32_t)(i % STAGES) * C::UNIT;
                const uint32_t dst = st + lane * 16, vdst = st + 2 * KJ * 512 + v_slot;
                if (ok && n0 + 16 <= end && D == DP) {
                    const uint8_t *const ksrc = a.c.k + base + k_off, *const vsrc = a.c.v + base + v_off;
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
            tc::cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < STAGES - 1; ++i) issue(i);

        // ---- Q: scaled rows as fragments in shared memory ----------------------------
        // a warp takes 32 / LR rows at a time, LR lanes with 8 channels each a row
        {
            constexpr int LR = DP / 8, RW = 32 / LR;
            const int rl = lane / LR, ch = 8 * (lane % LR);
            for (int r0 = w * RW; r0 < ROWS; r0 += NW * RW) {
                const int r = r0 + rl;
                const RowPlace p = row_place(a, cur.s, cur.b, cur.rt, cur.h, r);
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
                if (p.valid && ch < D) load_q8(a, !F32, p.q + ch, x);
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
                for (int y = LR / 2; y; y >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, y));
                const int e = imax((int)(top >> 23) - 127, -100);
                const float inv = __int_as_float((14 - e + 127) << 23);      // e <= 127: a normal number
                if (ch == 0) factor[r] = top >= 0x7f800000u ? NAN : __int_as_float((e - 14 + 127) << 23) * a.sl2;
                // channels ch .. ch + 7 of row r: two k-steps' shares of lane t'; see the layouts above
                const int j = ch >> 6, tt = (ch >> 4) & 3, ln = (r & 7) * 4 + tt;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const int s = ((ch >> 2) & 3) + (i >> 2), reg = ((i >> 1) & 1) * 2 + ((r & 15) >> 3);
                    const float y0 = x[i] * inv, y1 = x[i + 1] * inv;
                    const uint32_t q0 = pack_f16(y0, y1);
                    uint32_t *f = reinterpret_cast<uint32_t *>(smem + C::Q_OFF) +
                                  (((r >> 4) * C::PARTS) * KS + j * 4 + s) * 128 + ln * 4 + reg;
                    f[0] = q0;
                    if (F32) f[KS * 128] = pack_rest(y0, y1, q0);
                }
            }
        }
        __syncthreads();
        float c[MT][2], m[MT][2], l[MT][2];
        int lim[MT][2], min_lim = 0x7fffffff;
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = 16 * x + 8 * y + g;
                const RowPlace p = row_place(a, cur.s, cur.b, cur.rt, cur.h, r);
                c[x][y] = factor[r];
                m[x][y] = kNoMax;
                l[x][y] = 0.f;
                lim[x][y] = p.valid ? p.limit : end;
                min_lim = imin(min_lim, lim[x][y]);
            }
        min_lim = imin(__reduce_min_sync(0xffffffffu, min_lim), end);
        // one row tile of bf16: Q stays in registers (from shared memory it would be half of
        // the traffic there)
        constexpr bool QREG = !F32 && MT == 1;
        uint32_t qf[QREG ? KS : 1][4];
        if (QREG)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint4 v = lds16(sbase + C::Q_OFF + k * 512 + lane * 16);
                qf[k % (QREG ? KS : 1)][0] = v.x; qf[k % (QREG ? KS : 1)][1] = v.y;
                qf[k % (QREG ? KS : 1)][2] = v.z; qf[k % (QREG ? KS : 1)][3] = v.w;
            }
        float o[MT][NO][4];
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int j = 0; j < NO; ++j)
#pragma unroll
                for (int y = 0; y < 4; ++y) o[x][j][y] = 0.f;

        // ---- units --------------------------------------------------------------------
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            cp_wait<STAGES - 2>();
            const uint32_t st = ring + (uint32_t)(i % STAGES) * C::UNIT;
            float s[MT][2][4];
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int y = 0; y < 4; ++y) s[x][n][y] = 0.f;
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
                                for (int y = 0; y < 4; ++y) f[y] = qf[(j * 4 + q) % (QREG ? KS : 1)][y];
                            } else {
                                const uint4 v = lds16(sbase + C::Q_OFF + ((x * C::PARTS + part) * KS + j * 4 + q) * 512 + lane * 16);
                                f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
                            }
                            mma16816(s[x][0], f, a0, a1);
                            mma16816(s[x][1], f, b0, b1);
                        }
                }
            }
            const uint2 sc = lds8(st + C::UNIT - 256 + lane * 8);
            const float ks = __uint_as_float(sc.x), vs = __uint_as_float(sc.y);
            const float ev = (float)((int)(sc.y >> 23) - 127);
            const float inv_vs = __int_as_float((254 - (int)(sc.y >> 23)) << 23);
            const int n0 = (u0 + w + i * NW) * 16;
            const bool whole = vs != 0.f && n0 + 16 <= min_lim;
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
                        for (int z = 0; z < 4; ++z) {
                            const int n = n0 + 2 * t + (z & 1) + 8 * (z >> 1);
                            if (vs == 0.f || n >= lim[x][y] || n >= end) hidden |= 1u << z;
                        }
                    // exponents of the weights against reference `ref`: one rounding each
                    float u[4];
                    auto exponents = [&](float ref) {
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            u[z] = fmaf(v[z], cc, ev - ref);
                            if (hidden >> z & 1) u[z] = -INFINITY;
                        }
                        return fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3]));
                    };
                    if (__any_sync(0xffffffffu, exponents(m[x][y]) > kHeadroom)) {
                        float best = exponents(0.f);
                        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
                        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
                        if (best > m[x][y] + kHeadroom) {
                            const float f = tc::ex2(m[x][y] - (best - kFresh));
                            m[x][y] = best - kFresh;
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
                    for (int z = 0; z < 4; ++z) p[z] = tc::ex2(u[z]);
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
                        if (F32) mma16816(o[x][4 * q + j], pr[x], b0[j], b1[j]);
                        mma16816(o[x][4 * q + j], pf[x], b0[j], b1[j]);
                    }
            }
            issue(i + STAGES - 1);
        }
        cp_wait<0>();
        // ---- the warps' states become one -------------------------------------------------
        const int active = imin(NW, units);
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float v = l[x][y];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (t == 0) {
                    const int r = 16 * x + 8 * y + g;
                    m_sh[w * ROWS + r] = m[x][y];
                    l_sh[w * ROWS + r] = v;
                }
            }
        __syncthreads();                             // every warp is done with its ring
        const int rows = imin(ROWS, cur.s.n * a.G - cur.rt * ROWS);       // of this tile that are someone's
        if (w < active) {
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    if (16 * x + 8 * y + g < rows)
#pragma unroll
                    for (int j = 0; j < NO; ++j)
                        *reinterpret_cast<float2 *>(&join[(w * ROWS + 16 * x + 8 * y + g) * C::OS + 8 * j + 2 * t]) =
                            make_float2(o[x][j][2 * y], o[x][j][2 * y + 1]);
        }
        __syncthreads();
        const bool final = k0 == 0 && k1 == cur.nt;
        const int64_t slot = (int64_t)cta * 2 + (k0 == 0 ? 1 : 0);
        for (int i = tid; i < rows * (DP / 4); i += NT) {
            const int r = i / (DP / 4), d = (i % (DP / 4)) * 4;
            if (d >= D) continue;
            const RowPlace p = row_place(a, cur.s, cur.b, cur.rt, cur.h, r);
            float M = kNoMax;
            for (int x = 0; x < active; ++x) M = fmaxf(M, m_sh[x * ROWS + r]);
            float ls = 0.f;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            const int n = d / C::VB, j = d % C::VB;           // channel d = VB n + j
            for (int x = 0; x < active; ++x) {
                const float f = tc::ex2(m_sh[x * ROWS + r] - M);
                ls = fmaf(f, l_sh[x * ROWS + r], ls);
#pragma unroll
                for (int y = 0; y < 4; ++y) v[y] = fmaf(f, join[(x * ROWS + r) * C::OS + 8 * (j + y) + n], v[y]);
            }
            if (CL) {
                *reinterpret_cast<float4 *>(&ex_o[r * DP + d]) = make_float4(v[0], v[1], v[2], v[3]);
                if (d == 0) ex_ml[r] = make_float2(M, ls);
            } else if (final) {
                const float inv = ls == 0.f ? 0.f : 1.f / ls;
                store_o4(a, F32 || a.o_f32, p.o + d, make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
                if (a.L && d == 0) a.L[p.l] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(&a.part_O[(slot * a.rows + r) * D + d]) = make_float4(v[0], v[1], v[2], v[3]);
                if (d == 0) a.part_ml[slot * a.rows + r] = make_float2(M, ls);
            }
        }
        if (CL) {
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
                store_o4(a, F32 || a.o_f32, p.o + d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                if (a.L && d == 0) a.L[p.l] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * kLn2;
            }
            cluster_sync();                          // no block leaves while another reads it
            return;
        }
        __syncthreads();                             // the joining buffer is the next piece's ring
        cur.tiles_left -= k1 - k0;
        if (cur.tiles_left > 0) next_item(a, cur);
    }
    tc::pdl_launch_dependents();
}

template <int DP, int MT, bool F32, bool CL>
cudaError_t launch_as(const AttnArgs &a, int grid, int cluster, cudaStream_t st) {
    using C = MmaCfg<DP, MT, F32, CL>;
    auto k = attn_mma_kernel<DP, MT, F32, CL>;
    static SharedMemoryLimit limit;
    cudaError_t e = limit.raise((const void *)k, (int)C::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(C::NT);
    cfg.dynamicSmemBytes = C::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, k, a);
    note_launch();
    return e == cudaSuccess ? cudaGetLastError() : e;
}
template <int DP, int MT, bool F32>
cudaError_t launch_mma(const AttnArgs &a, int cluster, cudaStream_t st) {
    if (cluster > 1) {
        const int64_t items = (int64_t)a.c.B * a.c.H * row_tiles({0, a.n, 0, true}, a.G, a.rows);
        return launch_as<DP, MT, F32, true>(a, (int)items * cluster, cluster, st);
    }
    return launch_as<DP, MT, F32, false>(a, a.grid, 1, st);
}

}  // namespace

cudaError_t launch_attn_mma(const AttnArgs &a, bool bf16, int cluster, cudaStream_t st) {
    const bool wide = a.c.D > 64, two = a.rows == 32;
    if (bf16) {
        if (wide) return two ? launch_mma<128, 2, false>(a, cluster, st) : launch_mma<128, 1, false>(a, cluster, st);
        return two ? launch_mma<64, 2, false>(a, cluster, st) : launch_mma<64, 1, false>(a, cluster, st);
    }
    return wide ? launch_mma<128, 1, true>(a, cluster, st) : launch_mma<64, 1, true>(a, cluster, st);
}

}  // namespace cache
}  // namespace flare
