// K10: attention of one query token per sequence over a paged key-value cache.
//
// o = sum_j p_j v_j / sum_j p_j, p_j = exp(c q . k_j), over the kv_len tokens of the sequence; the
// G query heads of a key/value head read its rows together (up to 16 of them: one row group).
// Bound by reading K and V once.  One CTA per SM; the (sequence, row group, 64-token tile)
// units are counted in that order and cut into as many equal pieces as there are CTAs, so that
// every SM reads the same number of bytes whatever the lengths are.  A producer warp resolves pages
// and keeps a ring of tiles in flight (192 KB: TMA boxes of one page's rows, 128-byte swizzle);
// consumer warps keep the running maximum, sum and output of a segment (one row group's tiles
// inside the piece).  A segment that covers all of its item's tiles writes o; otherwise it
// leaves (m, l, O) in the workspace, and the last of an item's pieces to arrive joins them:
//   m = max_k m_k,  l = sum_k 2^{m_k - m} l_k,  o = sum_k 2^{m_k - m} O_k / l,
// always in the order of the pieces, so that the result does not depend on who comes last.
// Measured: 64 sequences of 1000-8000 tokens, 32/8 heads, d = 128, bf16: 148 us, 6.0 TB/s; 3 of 65536-131072, 8
// heads: 181 us, 6.5 TB/s; float32, 64 x 4000, 32/8 heads, d = 128: 319 us, 6.6 TB/s; d = 64, 64 x 8000, 16/8 heads,
// bf16: 172 us, 6.1 TB/s.  The producer's warp holds all nine to 168 registers a thread, and the kernels for
// d = 128 keep about 100 bytes of theirs in local memory (64 in float32, groups of up to 4).  Short calls are bound by their chain of dependent accesses (lengths, pages, first
// tile: 5 us; records, count, records read back where pieces are joined: 4 more: one sequence of 1000 tokens
// 9.3 us).
// Every wait is bounded (1 s, then LOLA_ATTN_TIMEOUT).
#include "lola_paged.cuh"

namespace lola {
namespace {

// ---- float32, CUDA cores ----
// Eight warps, the two halves of them on alternate tiles of a segment.  A warp takes four query rows and
// 64 / NP tokens of a tile (RM = 4, 8, 16 rows compiled for: NP = 4, 2, 1 parts of the tokens), 16 at a time,
// with its own running maximum, sum and output, joined at the segment's end: no barrier inside a segment (with
// all threads on one tile and two barriers in it, 64 sequences of 4000 tokens, 4 heads of 64, took 184 us, now 86).
// Lanes 8 tg + j: chunk j (16 bytes) of every 128-byte column of the rows, tokens 4 i + tg, so that K and V are
// read once, without bank conflicts, into products with q and the output in registers; the eight lanes' sums
// of a score are added and dealt out by halves (14 shuffles for 16 tokens x 4 rows).  m is the maximum so far:
// the largest weights' exponents stay near zero, where they lose least.
template <int D, int RM, bool SH, bool PRE>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_f32_kernel(const __grid_constant__ Maps maps, const Args a) {
    using C = Cfg<float, D>;
    constexpr int NC = RM / 4, NP = 4 / NC, KT = kTile / NP, X = D / 32, NW = kCons / kWarp;
    constexpr bool kHold = D == 64;                             // q in registers (168 a thread: nine warps)
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) Bars<C::kStages> bars;
    __shared__ uint32_t bad_sm[C::kStages];
    __shared__ int abort_sm, go;
    __shared__ Seg segs[1];
    __shared__ __align__(16) float Qs[kRows][D];
    __shared__ __align__(16) float Ps[NW][16][4];               // a warp's weights, to be read by token
    __shared__ __align__(16) float red[2 * NP][RM][D];          // the parts' outputs at a segment's end
    __shared__ float ms[2 * NP][RM], ls[2 * NP][RM];
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 1);
            mbar_init(smem_u32(&bars.empty[s]), NW / 2);
        }
        mbar_init(smem_u32(&bars.seg_full[0]), 1);
        mbar_init(smem_u32(&bars.seg_empty[0]), NW);
        abort_sm = 0;
        bars.issued = bars.ahead = bars.given = bars.arrived[0] = bars.arrived[1] = 0;
    }
    wait_for_last_kernel();
    Start st;
    if (!find_start<SH, kThreads, kTile, kRows, PRE>(a, &st)) return;
    if (warp == NW) produce<float, float, D, 1, SH, C, kRows, PRE>(maps, a, st, smem_u32(sm), smem_u32(Qs), D * 4, bars, segs, bad_sm, &abort_sm, lane);
    auto bar = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    const int grp = warp >> 2, rc = (warp & 3) / NP, tp = (warp & 3) % NP, tg = lane >> 3, j = lane & 7;
    const bool b2 = j & 4, b1 = j & 2, b0 = j & 1;
    const int box = min(p.page, kTile), lb = 31 - __clz(box);
    // byte offset of 16-byte chunk 0 of a token's row; column x (128 bytes) is x * box * 128 further
    auto row_at = [&](int k) { return (k >> lb) * box * C::kRowBytes + (k & (box - 1)) * 128; };
    for (int i = 0; warp < NW; ++i) {
        if (group_or<kCons>(1, !ring_wait(smem_u32(&bars.seg_full[0]), (uint32_t)i & 1, &abort_sm))) {
            if (tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
        const Seg g = segs[0];
        if (g.R < 0) break;
        if (!SH && !g.whole && tid == 64) open_cells<D>(a, g);
        auto q_at = [&](int r, int x) { return *reinterpret_cast<const float4*>(&Qs[4 * rc + r][32 * x + 4 * j]); };
        float4 q[4][kHold ? X : 1], acc[4][X];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int x = 0; x < X; ++x) {
                if (kHold) q[r][x] = q_at(r, x);
                acc[r][x] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        auto release = [&] {                                            // (g and the Q rows are in registers, or read)
            __syncwarp();
            if (lane == 0) mbar_arrive1(smem_u32(&bars.seg_empty[0]));
        };
        if (kHold) release();
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};         // rows 2 b0 and 2 b0 + 1
        bool ok = true;
        for (int t = (g.n0 ^ grp) & 1; t < g.tiles; t += 2) {
            const int n = g.n0 + t, s = n % C::kStages;
            ok = issued_wait(&bars.issued, n, &abort_sm) &&
                 ring_wait(smem_u32(&bars.full[s]), (uint32_t)(n / C::kStages) & 1, &abort_sm);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t* Kt = sm + (size_t)s * 2 * C::kHalf;
            uint8_t* Vt = Kt + C::kHalf;
            const uint32_t info = bad_sm[s], bad = PRE ? info & 0xffffu : info;
            const int nk = PRE ? (int)(info >> 16) : max(0, min(kTile, g.len - t * kTile));
            auto hidden = [&](int k) { return k >= nk || ((bad >> (k >> lb)) & 1u); };
            const bool some = nk < kTile || bad;
            if (some) {
                // tokens behind the sequence or on bad pages: their V rows (which may hold anything) become zero
                for (int k = tp * KT; k < (tp + 1) * KT; ++k)
                    if (hidden(k) && lane < D / 4)
                        *reinterpret_cast<float4*>(Vt + row_at(k) + (lane >> 3) * (box * 128) + (lane & 7) * 16) = make_float4(0.f, 0.f, 0.f, 0.f);
                fence_async_smem();            // (before the ring's next copy lands on these rows)
                __syncwarp();
            }
#pragma unroll 1
            for (int k0 = tp * KT; k0 < min((tp + 1) * KT, nk); k0 += 16) {
                // ---- scores of 16 tokens: this lane's channels ----
                const int at = row_at(k0) + tg * 128;
                float sc[4][4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[y][r] = 0.f;
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    float4 qx[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) qx[r] = kHold ? q[r][kHold ? x : 0] : q_at(r, x);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float4 k = *reinterpret_cast<const float4*>(Kt + at + x * (box * 128) + y * 512 + (((j ^ (4 * y + tg)) & 7) << 4));
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            sc[y][r] = fmaf(qx[r].w, k.w, fmaf(qx[r].z, k.z, fmaf(qx[r].y, k.y, fmaf(qx[r].x, k.x, sc[y][r]))));
                    }
                }
                // ---- added over the eight lanes: token 4 (j >> 1) + tg, rows 2 b0 and 2 b0 + 1 stay here ----
                float u[2][4], w[4], z[2];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        u[y][r] = (b2 ? sc[2 + y][r] : sc[y][r]) + __shfl_xor_sync(0xffffffffu, b2 ? sc[y][r] : sc[2 + y][r], 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r] = (b1 ? u[1][r] : u[0][r]) + __shfl_xor_sync(0xffffffffu, b1 ? u[0][r] : u[1][r], 2);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    z[e] = ((b0 ? w[2 + e] : w[e]) + __shfl_xor_sync(0xffffffffu, b0 ? w[e] : w[2 + e], 1)) * a.scale_log2;
                if (some && hidden(k0 + 4 * (j >> 1) + tg)) z[0] = z[1] = -INFINITY;
                // ---- running maximum, weights ----
                bool need[2];
                float bm[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    bm[e] = z[e];
#pragma unroll
                    for (int o = 2; o < kWarp; o <<= 1) bm[e] = fmaxf(bm[e], __shfl_xor_sync(0xffffffffu, bm[e], o));
                    need[e] = bm[e] > m[e];
                }
                if (__any_sync(0xffffffffu, need[0] || need[1])) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        f[e] = need[e] ? exp2f(m[e] - bm[e]) : 1.f;
                        if (need[e]) m[e] = bm[e];
                        l[e] *= f[e];
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float fr = __shfl_sync(0xffffffffu, f[r & 1], (lane & 30) | (r >> 1));
#pragma unroll
                        for (int x = 0; x < X; ++x) acc[r][x] = make_float4(acc[r][x].x * fr, acc[r][x].y * fr, acc[r][x].z * fr, acc[r][x].w * fr);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    z[e] = exp2f(z[e] - (m[e] == -INFINITY ? 0.f : m[e]));
                    l[e] += z[e];
                }
                *reinterpret_cast<float2*>(&Ps[warp][4 * (j >> 1) + tg][2 * (j & 1)]) = make_float2(z[0], z[1]);
                __syncwarp();
                // ---- O += P V ----
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float4 pr = *reinterpret_cast<const float4*>(&Ps[warp][4 * y + tg][0]);
                    const float pv[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        const float4 v = *reinterpret_cast<const float4*>(Vt + at + x * (box * 128) + y * 512 + (((j ^ (4 * y + tg)) & 7) << 4));
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            acc[r][x].x = fmaf(pv[r], v.x, acc[r][x].x);
                            acc[r][x].y = fmaf(pv[r], v.y, acc[r][x].y);
                            acc[r][x].z = fmaf(pv[r], v.z, acc[r][x].z);
                            acc[r][x].w = fmaf(pv[r], v.w, acc[r][x].w);
                        }
                    }
                }
                __syncwarp();                                           // (Ps is read)
            }
            if (lane == 0) mbar_arrive1(smem_u32(&bars.empty[s]));
        }
        // ---- the segment's end: the lanes' tokens (row tg stays here), then the parts in order ----
        if (group_or<kCons>(1, !ok)) {
            if (tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
        if (!kHold) release();
        const int part = grp * NP + tp;
        auto give = [](const float4& x, int o) {
            return make_float4(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o),
                               __shfl_xor_sync(0xffffffffu, x.z, o), __shfl_xor_sync(0xffffffffu, x.w, o));
        };
        auto plus = [](const float4& x, const float4& y) { return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); };
#pragma unroll
        for (int x = 0; x < X; ++x) {
            const bool t1 = tg & 2, t0 = tg & 1;
            const float4 y0 = plus(t1 ? acc[2][x] : acc[0][x], give(t1 ? acc[0][x] : acc[2][x], 16));
            const float4 y1 = plus(t1 ? acc[3][x] : acc[1][x], give(t1 ? acc[1][x] : acc[3][x], 16));
            const float4 y = plus(t0 ? y1 : y0, give(t0 ? y0 : y1, 8));
            *reinterpret_cast<float4*>(&red[part][4 * rc + tg][32 * x + 4 * j]) = y;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 2; o < kWarp; o <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
            if (lane < 2) {
                ms[part][4 * rc + 2 * lane + e] = m[e];
                ls[part][4 * rc + 2 * lane + e] = l[e];
            }
        }
        bar();
        float* rec = segment_record<D, SH>(a, g);
        for (int e = tid; e < g.R * (D / 4); e += kCons) {
            const int r = e / (D / 4), c = e % (D / 4) * 4;
            float M = -INFINITY, ll = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2 * NP; ++k) M = fmaxf(M, ms[k][r]);
#pragma unroll
            for (int k = 0; k < 2 * NP; ++k) {
                const float f = exp2f(ms[k][r] - (M == -INFINITY ? 0.f : M));
                const float4 x = *reinterpret_cast<const float4*>(&red[k][r][c]);
                ll = fmaf(f, ls[k][r], ll);
                y[0] = fmaf(f, x.x, y[0]);
                y[1] = fmaf(f, x.y, y[1]);
                y[2] = fmaf(f, x.z, y[2]);
                y[3] = fmaf(f, x.w, y[3]);
            }
            write_out<float, D, SH>(a, g, g.whole, rec, r, c, y, M, ll);
        }
        if (!SH && !g.whole) join_pieces<float, D, kCons>(a, g, tid, &go, bars.arrived, bar);
        bar();                                                  // red, ms, ls are read
    }
    __syncthreads();
    if (abort_sm) settle<D, C::kStages, 1, SH, kThreads, kTile, PRE>(a, bars);
}

// ---- bf16: the tile products on the warps' matrix instructions ----
// Two groups of four warps: at d = 128 they take the segments in turn, so that one group's epilogue runs beside
// the other's tiles (64 sequences of 1000-8000 tokens, 32/8 heads, when both were built: 142 us, 152 on tiles in
// turn); at d = 64, where a tile's bytes come faster than four warps get through it, they take a segment's tiles in
// turn (64 x 8000 tokens, 16/8 heads, likewise: 171 us, 214 on segments in turn).  A warp takes 16 of a tile's 64 tokens, with its own running
// maximum, sum and output of the 16 query rows, joined at the segment's end.  S = Q K^T has the rows of Q as M, so
// that its accumulators are the A operand of P V as they stand.  m is raised lazily (it is set 8 above a
// maximum, so that no weight is above one), which leaves the output alone for most tiles.
template <int D, bool HALF> struct MmaSmem {
    static constexpr bool kBoth = D == 64;
    static constexpr int NW = kBoth ? 8 : 4;                                // warps of a segment
    static constexpr int HR = HALF ? 1 : 2, R8 = 8 * HR, CK = 512 / R8;     // rows kept; columns joined at a time
    static constexpr int kPitch = 2 * D + 16;                               // Q rows (16-byte shift against bank conflicts)
    float red[8 / NW][NW][R8][CK];                                               // by group and warp
    float ms[8 / NW][NW][R8], ls[8 / NW][NW][R8];
    uint8_t q[2][kRows * kPitch];
};

// HALF: at most 8 query rows (rows 8-15 of the products hold anything and are left alone)
template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_mma_kernel(const __grid_constant__ Maps maps, const Args a) {
    using T = __nv_bfloat16;
    using C = Cfg<T, D>;
    using M = MmaSmem<D, HALF>;
    constexpr int HR = M::HR, CK = M::CK;
    constexpr bool kBoth = M::kBoth;
    constexpr int NW = M::NW, NT = NW * kWarp;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    __shared__ __align__(16) M x;
    __shared__ __align__(8) Bars<C::kStages> bars;
    __shared__ uint32_t bad_sm[C::kStages];
    __shared__ int abort_sm, go[2];
    __shared__ Seg segs[2];
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 1);
            mbar_init(smem_u32(&bars.empty[s]), 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars.seg_full[s]), 1);
            mbar_init(smem_u32(&bars.seg_empty[s]), NW);
        }
        abort_sm = 0;
        bars.issued = bars.ahead = bars.given = bars.arrived[0] = bars.arrived[1] = 0;
    }
    wait_for_last_kernel();
    Start st;
    if (!find_start<false>(a, &st)) return;
    if (warp == kCons / kWarp) produce<T, T, D, 2, false>(maps, a, st, sb, smem_u32(x.q[0]), M::kPitch, bars, segs, bad_sm, &abort_sm, lane);
    const int grp = warp >> 2, wg = warp & 3, g8 = lane >> 2, q2 = (lane & 3) * 2;
    const int own = kBoth ? 0 : grp, me = kBoth ? warp : wg, gt = kBoth ? tid : tid & 127;   // the segment's group, its warps and threads
    auto bar = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + own), "n"(NT) : "memory"); };
    const int k0 = wg * 16;                                            // this warp's tokens of a tile
    const int box = min(p.page, kTile), lb = 31 - __clz(box);
    const uint32_t col = (uint32_t)box * 128;                          // from one 128-byte column to the next
    auto row_at = [&](int k) { return (uint32_t)((k >> lb) * box * C::kRowBytes + (k & (box - 1)) * 128); };
    const int kkey = k0 + ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;        // ldmatrix rows of K
    const int vkey = k0 + (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;        // ... of V
    const uint32_t krow = row_at(kkey), vrow = C::kHalf + row_at(vkey);
    const uint32_t qrow = smem_u32(x.q[0]) + ((lane & 7) + ((lane >> 3) & 1) * 8) * M::kPitch + (lane >> 4) * 16;
    for (int i = 0; warp < kCons / kWarp; ++i) {
        const int slot = kBoth ? i & 1 : grp;
        if (group_or<NT>(1 + own, !ring_wait(smem_u32(&bars.seg_full[slot]), (uint32_t)(kBoth ? i >> 1 : i) & 1, &abort_sm))) {
            if (gt == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
        const Seg g = segs[slot];
        if (g.R < 0) break;
        if (!g.whole && gt == 64) open_cells<D>(a, g);
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int y = 0; y < D / 16; ++y) ldsm4(qrow + slot * kRows * M::kPitch + 32 * y, qa[y]);
        __syncwarp();
        if (lane == 0) mbar_arrive1(smem_u32(&bars.seg_empty[slot]));   // (g and the Q rows are in registers)
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[y][e] = 0.f;
        bool ok = true;
        for (int t = kBoth ? (g.n0 ^ grp) & 1 : 0; t < g.tiles; t += kBoth ? 2 : 1) {
            const int n = g.n0 + t, s = n % C::kStages;
            ok = issued_wait(&bars.issued, n, &abort_sm) &&
                 ring_wait(smem_u32(&bars.full[s]), (uint32_t)(n / C::kStages) & 1, &abort_sm);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t kt = sb + (uint32_t)s * 2 * C::kHalf;
            const int left = g.len - t * kTile;
            const uint32_t bad = bad_sm[s];
            // ---- S: 16 rows x 16 tokens, two chains a token half ----
            float c0[2][4] = {}, c1[2][4] = {};
#pragma unroll
            for (int y = 0; y < D / 16; ++y) {
                uint32_t kb[4];
                const int ch = 2 * y + kch;
                ldsm4(kt + krow + (ch >> 3) * col + (((ch ^ kkey) & 7) << 4), kb);
                mma16816(y & 1 ? c1[0] : c0[0], qa[y], kb[0], kb[1]);
                mma16816(y & 1 ? c1[1] : c0[1], qa[y], kb[2], kb[3]);
            }
            float sc[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[y][e] = c0[y][e] + c1[y][e];
            if (left < k0 + 16 || bad) {
                // tokens behind the sequence or on bad pages: no score, and their V rows (which may
                // hold anything) become zero
                const int nk = max(0, min(kTile, left));
                auto hidden = [&](int k) { return k >= nk || ((bad >> (k >> lb)) & 1u); };
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hidden(k0 + 8 * y + q2 + (e & 1))) sc[y][e] = -INFINITY;
                for (int k = k0; k < k0 + 16; ++k)
                    if (hidden(k) && lane < D / 8)
                        *reinterpret_cast<uint4*>(sm + (size_t)s * 2 * C::kHalf + C::kHalf + row_at(k) + (lane >> 3) * col +
                                                  (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();            // (before the ring's next copy lands on these rows)
                __syncwarp();
            }
            // ---- running maximum, weights ----
            uint32_t pa[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int r = 0; r < HR; ++r) {
                float bm = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                const float top = fmaf(fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2)), a.scale_log2, kRaise);
                const bool need = top > m[r] + kRaise;
                if (__any_sync(0xffffffffu, need)) {
                    const float f = need ? ex2(m[r] - top) : 1.f;
                    if (need) m[r] = top;
                    l[r] *= f;
#pragma unroll
                    for (int y = 0; y < D / 8; ++y) {
                        o[y][2 * r] *= f;
                        o[y][2 * r + 1] *= f;
                    }
                }
                const float base = m[r] == -INFINITY ? 0.f : m[r];
                const float e0 = ex2(fmaf(sc[0][2 * r], a.scale_log2, -base)), e1 = ex2(fmaf(sc[0][2 * r + 1], a.scale_log2, -base));
                const float e2 = ex2(fmaf(sc[1][2 * r], a.scale_log2, -base)), e3 = ex2(fmaf(sc[1][2 * r + 1], a.scale_log2, -base));
                l[r] += (e0 + e1) + (e2 + e3);
                pa[r] = pack2(e0, e1);
                pa[2 + r] = pack2(e2, e3);
            }
            // ---- O += P V ----
#pragma unroll
            for (int y = 0; y < D / 16; ++y) {
                uint32_t vb[4];
                const int ch = 2 * y + vch;
                ldsm4_t(kt + vrow + (ch >> 3) * col + (((ch ^ vkey) & 7) << 4), vb);
                mma16816(o[2 * y], pa, vb[0], vb[1]);
                mma16816(o[2 * y + 1], pa, vb[2], vb[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(smem_u32(&bars.empty[s]));
        }
        // ---- the segment's end: add the warps in order, then o or the piece's record ----
        if (group_or<NT>(1 + own, !ok)) {
            if (gt == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if ((lane & 3) == 0) {
                x.ms[own][me][g8 + 8 * r] = m[r];
                x.ls[own][me][g8 + 8 * r] = l[r];
            }
        }
        bar();
        float f[2];
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < NW; ++w) mm = fmaxf(mm, x.ms[own][w][g8 + 8 * r]);
            f[r] = ex2(m[r] - (mm == -INFINITY ? 0.f : mm));
        }
        float* rec = segment_record<D, false>(a, g);
        const int er = 4 * (gt & 127) / CK, ec = 4 * (gt & 127) % CK;        // 128 threads x 4 columns = R8 x CK
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, x.ms[own][w][er]);
#pragma unroll
        for (int w = 0; w < NW; ++w) ll = fmaf(x.ls[own][w][er], ex2(x.ms[own][w][er] - (mm == -INFINITY ? 0.f : mm)), ll);
#pragma unroll
        for (int c = 0; c < D; c += CK) {
            if (c > 0) bar();
#pragma unroll
            for (int y = 0; y < CK / 8; ++y)
#pragma unroll
                for (int r = 0; r < HR; ++r)
                    *reinterpret_cast<float2*>(&x.red[own][me][g8 + 8 * r][8 * y + q2]) =
                        make_float2(o[c / 8 + y][2 * r] * f[r], o[c / 8 + y][2 * r + 1] * f[r]);
            bar();
            if (!kBoth || gt < 128) {
                float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float4 z = *reinterpret_cast<const float4*>(&x.red[own][w][er][ec]);
                    y[0] += z.x;
                    y[1] += z.y;
                    y[2] += z.z;
                    y[3] += z.w;
                }
                if (er < g.R) write_out<T, D, false>(a, g, g.whole, rec, er, c + ec, y, mm, ll);
            }
        }
        if (!g.whole) join_pieces<T, D, NT>(a, g, gt, &go[own], bars.arrived, bar);
    }
    __syncthreads();
    if (abort_sm) settle<D, C::kStages, 2, false>(a, bars);
}

// (rows of a prefix: as many as its sequences have)
template <int D, bool SH, bool PRE = false>
cudaError_t launch_f32(const DecodeArgs& d, cudaStream_t st) {
    static std::atomic<uint64_t> done[3] = {};
    const int rows = !SH || d.sh.each ? d.p.G : kRows;
    if (rows <= 4) return launch_kernel<float, D>(paged_decode_f32_kernel<D, 4, SH, PRE>, kThreads / kWarp, done[0], d, st);
    if (rows <= 8) return launch_kernel<float, D>(paged_decode_f32_kernel<D, 8, SH, PRE>, kThreads / kWarp, done[1], d, st);
    return launch_kernel<float, D>(paged_decode_f32_kernel<D, 16, SH, PRE>, kThreads / kWarp, done[2], d, st);
}
template <int D>
cudaError_t launch_bf16(const DecodeArgs& d, cudaStream_t st) {
    static std::atomic<uint64_t> done[2] = {};
    return d.p.G <= 8 ? launch_kernel<__nv_bfloat16, D>(paged_decode_mma_kernel<D, true>, kThreads / kWarp, done[0], d, st)
                      : launch_kernel<__nv_bfloat16, D>(paged_decode_mma_kernel<D, false>, kThreads / kWarp, done[1], d, st);
}

}  // namespace

int64_t paged_decode_workspace(int d) { return (int64_t)kPieces * kSlots * (record_floats(d) * sizeof(float) + sizeof(uint64_t)); }

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_f32<128, false>(a, st) : launch_f32<64, false>(a, st);
    return a.p.d == 128 ? launch_bf16<128>(a, st) : launch_bf16<64>(a, st);
}
cudaError_t launch_f32_parts(const DecodeArgs& a, cudaStream_t st) {
    return a.p.d == 128 ? launch_f32<128, true>(a, st) : launch_f32<64, true>(a, st);
}
cudaError_t launch_f32_behind(const DecodeArgs& a, cudaStream_t st) {
    return a.p.d == 128 ? launch_f32<128, false, true>(a, st) : launch_f32<64, false, true>(a, st);
}

cudaError_t paged_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
