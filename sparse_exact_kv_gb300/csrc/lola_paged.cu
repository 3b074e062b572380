// K10: attention of one query token per sequence over a paged key-value cache.
//
// o = sum_j p_j v_j / sum_j p_j, p_j = exp(c q . k_j), over the kv_len tokens of the sequence; the
// G query heads of a key/value head read its rows together (up to 16 of them: one row group).
// Bound by reading K and V once.  One CTA per SM; the (sequence, row group, 64-token tile)
// units are counted in that order and cut into as many equal pieces as there are CTAs, so that
// every SM reads the same number of bytes whatever the lengths are.  A producer warp resolves pages
// and keeps a ring of tiles in flight (TMA boxes of one page's rows, 128-byte swizzle); eight
// consumer warps keep the running maximum, sum and output of the row group.  A piece that
// covers all of a sequence's tiles writes o; otherwise it leaves (m, l, O) in the workspace,
// where a second kernel joins the pieces in order:
//   m = max_k m_k,  l = sum_k 2^{m_k - m} l_k,  o = sum_k 2^{m_k - m} O_k / l.
// Every wait is bounded (1 s, then LOLA_ATTN_TIMEOUT).
#include <cuda.h>

#include "lola_attn.cuh"
#include "lola_tc.cuh"

namespace lola {
namespace {

using namespace tc;

__device__ int32_t g_status;

constexpr int kTile = 64;                 // tokens per tile
constexpr int kCons = 256;                // consumer threads
constexpr int kThreads = kCons + kWarp;
constexpr int kPieces = 152;              // one CTA per SM
constexpr int kRows = 16;                 // query rows of a row group (at most)
constexpr uint64_t kWaitNs = 1000000000ull;

struct Maps {
    CUtensorMap k, v;   // [n_pages * Hkv][page][d], boxes of 128 bytes x min(page, 64) rows
};

struct Args {
    PagedArgs p;
    Rows Q, O;
    float* lse;
    float* part;        // [kPieces][2][kRows][d + 2]: O, then m, l
    float scale_log2;
    int RG, I;          // row groups per key/value head; items (row groups) per sequence
};

template <typename T, int D> struct Cfg {
    static constexpr int kBoxes = D * (int)sizeof(T) / 128;        // 128-byte columns of a row
    static constexpr int kHalf = kTile * D * (int)sizeof(T);       // K or V of a tile
    static constexpr int kStages = 196608 / (2 * kHalf) > 8 ? 8 : 196608 / (2 * kHalf);
};

// Tiles of sequence b, for each of its items: at least one, so that an empty sequence's output
// is written too.
__device__ __forceinline__ int tiles_of(const PagedArgs& p, int b) {
    const int64_t n = paged_tokens(p, p.kv_len[b]);
    return n <= 0 ? 1 : (int)((n + kTile - 1) / kTile);
}

// Pieces of `total` units: none is empty.
__device__ __forceinline__ int pieces_of(int64_t total) { return (int)min((int64_t)kPieces, total); }

// The walk of one piece over its (sequence, item, tiles) segments, the same for every role.
struct Walk {
    int64_t left;         // units of the piece not yet walked
    int b, item, tiles, t0, t1;
    __device__ __forceinline__ void start(const PagedArgs& p, int I, int b_, int64_t rem, int64_t units) {
        b = b_;
        tiles = tiles_of(p, b);
        item = (int)(rem / tiles);
        t0 = (int)(rem % tiles);
        left = units;
        clip();
    }
    __device__ __forceinline__ void clip() { t1 = (int)min((int64_t)tiles, t0 + left); }
    __device__ __forceinline__ bool next(const PagedArgs& p, int I) {
        left -= t1 - t0;
        if (left <= 0) return false;
        t0 = 0;
        if (++item == I) {
            item = 0;
            ++b;
            tiles = tiles_of(p, b);
        }
        clip();
        return true;
    }
};

__device__ __forceinline__ void cons_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ float to_float(float x) { return x; }

template <typename T>
__device__ __forceinline__ void chunk_floats(const uint8_t* p, float (&v)[16 / sizeof(T)]) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, int* abort_sm) {
    uint64_t start = 0;
    for (int it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*reinterpret_cast<volatile int*>(abort_sm)) return false;
        const uint64_t now = globaltimer_ns();
        if (it == 0) start = now;
        else if (now - start > kWaitNs) {
            *abort_sm = 1;
            return false;
        }
    }
}

// The producer warp: the tiles of the piece's segments, in order, into the ring at `sb`.  A tile's
// pages outside the cache are not loaded; bit x of bad_sm marks the tile's x-th token box.
template <typename T, int D>
__device__ __forceinline__ void produce(const Maps& maps, const Args& a, Walk w, uint32_t sb, uint64_t* bars,
                                        uint32_t* bad_sm, int* abort_sm, int lane) {
    using C = Cfg<T, D>;
    const PagedArgs& p = a.p;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[C::kStages + s]); };
    const int box = min(p.page, kTile), nbox = kTile / box;   // token boxes of a tile
    const uint32_t row_bytes = D * sizeof(T);
    int64_t n = 0;
    bool ok = true;
    do {
        const int hk = w.item / a.RG;
        const int64_t len = paged_tokens(p, p.kv_len[w.b]);
        if (lane == 0 && p.kv_len[w.b] > len && len > 0) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
        int64_t base = -1;         // first of the 32 page-table columns the lanes hold
        int held = -1;
        for (int t = w.t0; t < w.t1 && ok; ++t, ++n) {
            const int s = (int)(n % C::kStages);
            if (n >= C::kStages) ok = __all_sync(0xffffffffu, ring_wait(empty(s), (uint32_t)((n / C::kStages) - 1) & 1, abort_sm));
            if (!ok) break;
            uint32_t bad = 0, bytes = 0;
            for (int x = 0; x < nbox; ++x) {
                const int64_t pos = (int64_t)t * kTile + x * box;
                if (pos >= len) break;
                const int64_t col = pos >> p.page_log2;
                if (base < 0 || col >= base + 32) {
                    base = col;
                    const int64_t c = base + lane;
                    held = (c << p.page_log2) < len ? paged_page(p, w.b, c << p.page_log2) : 0;
                }
                const int page = __shfl_sync(0xffffffffu, held, (int)(col - base));
                if (page < 0) bad |= 1u << x;
                else bytes += 2u * box * row_bytes;
            }
            if (lane == 0) {
                if (bad) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
                bad_sm[s] = bad;
                mbar_expect(full(s), bytes);
            }
            __syncwarp();
            for (int x = 0; x < nbox; ++x) {
                const int64_t pos = (int64_t)t * kTile + x * box;
                if (pos >= len) break;
                const int page = __shfl_sync(0xffffffffu, held, (int)((pos >> p.page_log2) - base));
                if (page < 0) continue;
                if (lane < 2 * C::kBoxes) {
                    const int c = lane % C::kBoxes, kv = lane / C::kBoxes;
                    const uint32_t dst = sb + (uint32_t)s * 2 * C::kHalf + kv * C::kHalf + c * (kTile * 128) + x * box * 128;
                    tma_load3(dst, kv ? &maps.v : &maps.k, c * (128 / (int)sizeof(T)), (int)(pos & (p.page - 1)),
                              page * p.Hkv + hk, full(s));
                }
            }
        }
    } while (ok && w.next(p, a.I));
    // leave no copy in flight
    if (lane == 0)
        for (int64_t i = n > C::kStages ? n - C::kStages : 0; i < n; ++i)
            mbar_wait(full((int)(i % C::kStages)), (uint32_t)(i / C::kStages) & 1, kWaitNs);
}

template <typename T, int D, int RM>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_kernel(const __grid_constant__ Maps maps, const Args a) {
    using C = Cfg<T, D>;
    constexpr int VN = 16 / (int)sizeof(T), CH = D / VN, KP = kCons / D;   // chunks a row; key parts of P V
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    __shared__ __align__(8) uint64_t bars[2 * C::kStages];
    __shared__ uint32_t bad_sm[C::kStages];
    __shared__ int abort_sm;
    __shared__ int64_t scan[kThreads / kWarp];
    __shared__ __align__(16) float Qs[RM][D];
    __shared__ __align__(16) float Ss[2][RM][kTile];
    __shared__ float fs[2][RM], ms[RM], ls[RM];
    __shared__ float red[KP - 1][RM][D];
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[C::kStages + s]); };
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kCons / kWarp);
        }
        abort_sm = 0;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto count = [&](int b) -> int64_t { return (int64_t)tiles_of(p, b) * a.I; };
    const int64_t total = seq_total<kThreads>(p.n_seq, count, scan);
    const int N = pieces_of(total);
    if ((int)blockIdx.x >= N) return;
    const int64_t u0 = split_at(total, N, blockIdx.x), u1 = split_at(total, N, blockIdx.x + 1);
    int b0;
    int64_t rem;
    seq_find<kThreads>(p.n_seq, count, u0, scan, &b0, &rem);
    Walk w;
    w.start(p, a.I, b0, rem, u1 - u0);

    if (warp == kCons / kWarp) {
        produce<T, D>(maps, a, w, sb, bars, bad_sm, &abort_sm, lane);
    } else {
        // ============================ consumers ============================
        const int key = tid % kTile, hs = tid / kTile;      // scores: one key, rows hs, hs + 4, ..
        const int dim = tid % D, part = tid / D;            // P V: one channel, keys of one part
        int64_t n = 0;
        bool ok = true;
        do {
            const int hk = w.item / a.RG, h0 = hk * p.G + (w.item % a.RG) * kRows;
            const int R = min(kRows, p.G - (w.item % a.RG) * kRows);
            const int64_t len = paged_tokens(p, p.kv_len[w.b]);
            cons_sync();                                    // the last segment's Qs, ms, ls are read
            for (int i = tid; i < RM * D; i += kCons) {
                const int r = i / D, c = i % D;
                const T* q = reinterpret_cast<const T*>(a.Q.data) + (int64_t)w.b * a.Q.row + (int64_t)(h0 + r) * a.Q.head;
                Qs[r][c] = r < R ? to_float(q[c]) * a.scale_log2 : 0.f;
            }
            if (tid < RM) {
                ms[tid] = -INFINITY;
                ls[tid] = 0.f;
            }
            float acc[RM];
#pragma unroll
            for (int r = 0; r < RM; ++r) acc[r] = 0.f;
            cons_sync();
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const int s = (int)(n % C::kStages), e = (int)(n & 1);
                if (ok) ok = ring_wait(full(s), (uint32_t)(n / C::kStages) & 1, &abort_sm);
                const uint8_t* Kt = sm + (size_t)s * 2 * C::kHalf;
                const uint8_t* Vt = Kt + C::kHalf;
                const int nk = (int)max((int64_t)0, min((int64_t)kTile, len - (int64_t)t * kTile));
                const uint32_t bad = ok ? bad_sm[s] : ~0u;
                const int box = min(p.page, kTile);
                // ---- scores ----
                float sc[(RM + 3) / 4];
#pragma unroll
                for (int i = 0; i < (RM + 3) / 4; ++i) sc[i] = 0.f;
                const bool seen = key < nk && !((bad >> (key / box)) & 1u);
#pragma unroll 4
                for (int c = 0; c < CH; ++c) {
                    float kv[VN];
                    chunk_floats<T>(Kt + (c / 8) * (kTile * 128) + key * 128 + (((c ^ key) & 7) << 4), kv);
#pragma unroll
                    for (int i = 0; i < (RM + 3) / 4; ++i) {
                        const int r = hs + 4 * i;
                        if (r < RM)
#pragma unroll
                            for (int x = 0; x < VN; ++x) sc[i] = fmaf(Qs[r][c * VN + x], kv[x], sc[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < (RM + 3) / 4; ++i)
                    if (hs + 4 * i < RM) Ss[e][hs + 4 * i][key] = seen ? sc[i] : -INFINITY;
                cons_sync();
                // ---- running maximum and sum: warp w takes rows w, w + 8 ----
                for (int r = warp; r < RM; r += kCons / kWarp) {
                    const float x = Ss[e][r][lane], y = Ss[e][r][lane + 32];
                    const float mo = ms[r], mn = fmaxf(mo, warp_max(fmaxf(x, y)));
                    const float bs = mn == -INFINITY ? 0.f : mn;
                    const float px = exp2f(x - bs), py = exp2f(y - bs);
                    const float f = exp2f(mo - bs), sum = warp_sum(px + py);
                    Ss[e][r][lane] = px;
                    Ss[e][r][lane + 32] = py;
                    __syncwarp();
                    if (lane == 0) {
                        ms[r] = mn;
                        ls[r] = ls[r] * f + sum;
                        fs[e][r] = f;
                    }
                }
                cons_sync();
                // ---- O += P V ----
#pragma unroll
                for (int r = 0; r < RM; ++r) acc[r] *= fs[e][r];
                constexpr int KN = kTile / KP;
                const uint32_t vcol = (dim * (int)sizeof(T)) % 128;
                const uint8_t* vb = Vt + (dim * (int)sizeof(T) / 128) * (kTile * 128) + (vcol & 15);
                for (int k4 = part * KN; k4 < min(nk, (part + 1) * KN); k4 += 4) {
                    float v[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int kk = k4 + x;
                        // (a key that is not seen has p = 0; its value row may be anything)
                        const bool in = kk < nk && !((bad >> (kk / box)) & 1u);
                        v[x] = in ? to_float(*reinterpret_cast<const T*>(vb + kk * 128 + ((((vcol >> 4) ^ kk) & 7) << 4))) : 0.f;
                    }
#pragma unroll
                    for (int r = 0; r < RM; ++r) {
                        const float4 pr = *reinterpret_cast<const float4*>(&Ss[e][r][k4]);
                        acc[r] = fmaf(pr.x, v[0], acc[r]);
                        acc[r] = fmaf(pr.y, v[1], acc[r]);
                        acc[r] = fmaf(pr.z, v[2], acc[r]);
                        acc[r] = fmaf(pr.w, v[3], acc[r]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive1(empty(s));
            }
            // ---- the segment's end: join the key parts, then o or the piece's (O, m, l) ----
            if (KP > 1) {
                if (part > 0)
#pragma unroll
                    for (int r = 0; r < RM; ++r) red[part - 1][r][dim] = acc[r];
                cons_sync();
                if (part == 0)
#pragma unroll
                    for (int r = 0; r < RM; ++r)
#pragma unroll
                        for (int k = 0; k < KP - 1; ++k) acc[r] += red[k][r][dim];
            }
            if (part == 0) {
                const bool whole = w.t0 == 0 && w.t1 == w.tiles;
                if (whole) {
                    T* o = reinterpret_cast<T*>(a.O.data) + (int64_t)w.b * a.O.row + (int64_t)h0 * a.O.head + dim;
#pragma unroll
                    for (int r = 0; r < RM; ++r)
                        if (r < R) {
                            const bool none = ls[r] == 0.f;
                            IO<T>::st(o, r * a.O.head, none ? 0.f : acc[r] / ls[r]);
                            if (a.lse && dim == 0)
                                a.lse[(int64_t)w.b * p.Hq + h0 + r] = none ? -INFINITY : (ms[r] + log2f(ls[r])) * kAttnLn2;
                        }
                } else {
                    // slot 0: the piece's first segment
                    float* o = a.part + ((int64_t)blockIdx.x * 2 + (w.left == u1 - u0 ? 0 : 1)) * kRows * (D + 2);
#pragma unroll
                    for (int r = 0; r < RM; ++r)
                        if (r < R) {
                            o[r * (D + 2) + dim] = acc[r];
                            if (dim == 0) {
                                o[r * (D + 2) + D] = ms[r];
                                o[r * (D + 2) + D + 1] = ls[r];
                            }
                        }
                }
            }
        } while (w.next(p, a.I));
        if (!ok && tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
    }
}

// ---- bf16: the tile products on the warps' matrix instructions ----
// A warp takes 16 of a tile's 64 tokens (warps 0-3 the even tiles, 4-7 the odd ones), with its own
// running maximum, sum and output of the 16 query rows, joined at the segment's end.  S = Q K^T has
// the rows of Q as M, so that its accumulators are the A operand of P V as they stand.  m is
// raised lazily (by more than 2^8 at a time), which leaves the output alone for most tiles.
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
constexpr float kRaise = 8.0f;

// HALF: at most 8 query rows (rows 8-15 of the products are zero and left alone)
template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_mma_kernel(const __grid_constant__ Maps maps, const Args a) {
    using T = __nv_bfloat16;
    using C = Cfg<T, D>;
    constexpr int NW = kCons / kWarp, HR = HALF ? 1 : 2, R8 = 8 * HR, CK = HALF ? 64 : 32;   // join: CK columns at a time
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    __shared__ __align__(8) uint64_t bars[2 * C::kStages];
    __shared__ uint32_t bad_sm[C::kStages];
    __shared__ int abort_sm;
    __shared__ int64_t scan[kThreads / kWarp];
    __shared__ __align__(16) float red[NW][R8][CK];
    __shared__ float ms[NW][R8], ls[NW][R8];
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bars[s]), 1);
            mbar_init(smem_u32(&bars[C::kStages + s]), NW / 2);
        }
        abort_sm = 0;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto count = [&](int b) -> int64_t { return (int64_t)tiles_of(p, b) * a.I; };
    const int64_t total = seq_total<kThreads>(p.n_seq, count, scan);
    const int N = pieces_of(total);
    if ((int)blockIdx.x >= N) return;
    const int64_t u0 = split_at(total, N, blockIdx.x), u1 = split_at(total, N, blockIdx.x + 1);
    int b0;
    int64_t rem;
    seq_find<kThreads>(p.n_seq, count, u0, scan, &b0, &rem);
    Walk w;
    w.start(p, a.I, b0, rem, u1 - u0);
    if (warp == NW) {
        produce<T, D>(maps, a, w, sb, bars, bad_sm, &abort_sm, lane);
        return;
    }
    const int grp = warp >> 2, g = lane >> 2, q2 = (lane & 3) * 2;
    const int k0 = (warp & 3) * 16;                                    // this warp's tokens of a tile
    const int kkey = k0 + ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;        // ldmatrix rows of K
    const int vkey = k0 + (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;        // ... of V
    const int box = min(p.page, kTile);
    int64_t n = 0;
    bool ok = true;
    do {
        const int hk = w.item / a.RG, h0 = hk * p.G + (w.item % a.RG) * kRows;
        const int R = min(kRows, p.G - (w.item % a.RG) * kRows);
        const int64_t len = paged_tokens(p, p.kv_len[w.b]);
        // Q as the A operand: rows g, g + 8 (zero behind the group)
        uint32_t qa[D / 16][4];
        const T* Q = reinterpret_cast<const T*>(a.Q.data) + (int64_t)w.b * a.Q.row + (int64_t)h0 * a.Q.head + q2;
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = g + 8 * (e & 1);
                qa[x][e] = r < R ? *reinterpret_cast<const uint32_t*>(Q + r * a.Q.head + x * 16 + 8 * (e >> 1)) : 0u;
            }
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][e] = 0.f;
        for (int t = w.t0; t < w.t1; ++t, ++n) {
            if ((int)(n & 1) != grp) continue;
            const int s = (int)(n % C::kStages);
            if (ok) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars[s]), (uint32_t)(n / C::kStages) & 1, &abort_sm));
            if (!ok) continue;
            const uint32_t kt = sb + (uint32_t)s * 2 * C::kHalf, vt = kt + C::kHalf;
            const int64_t left = len - (int64_t)t * kTile;
            const uint32_t bad = bad_sm[s];
            // ---- S: 16 rows x 16 tokens, two chains a token half ----
            float c0[2][4] = {}, c1[2][4] = {};
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                uint32_t kb[4];
                const int ch = 2 * x + kch;
                ldsm4(kt + (ch >> 3) * (kTile * 128) + kkey * 128 + (((ch ^ kkey) & 7) << 4), kb);
                mma16816(x & 1 ? c1[0] : c0[0], qa[x], kb[0], kb[1]);
                mma16816(x & 1 ? c1[1] : c0[1], qa[x], kb[2], kb[3]);
            }
            float sc[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[x][e] = c0[x][e] + c1[x][e];
            if (left < k0 + 16 || bad) {
                // tokens behind the sequence or on bad pages: no score, and their V rows (which may
                // hold anything) become zero
                const int nk = (int)max((int64_t)0, min((int64_t)kTile, left));
                auto hidden = [&](int k) { return k >= nk || ((bad >> (k / box)) & 1u); };
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hidden(k0 + 8 * x + q2 + (e & 1))) sc[x][e] = -INFINITY;
                for (int k = k0; k < k0 + 16; ++k)
                    if (hidden(k))
                        for (int ch = lane; ch < D / 8; ch += 32)
                            *reinterpret_cast<uint4*>(sm + (size_t)s * 2 * C::kHalf + C::kHalf + (ch >> 3) * (kTile * 128) +
                                                      k * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();            // (before the ring's next copy lands on these rows)
                __syncwarp();
            }
            // ---- running maximum, weights ----
            uint32_t pa[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int r = 0; r < HR; ++r) {
                float bm = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2)) * a.scale_log2;
                const bool need = bm > m[r] + kRaise || (m[r] == -INFINITY && bm > m[r]);
                if (__any_sync(0xffffffffu, need)) {
                    const float f = need ? ex2(m[r] - bm) : 1.f;
                    if (need) m[r] = bm;
                    l[r] *= f;
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) {
                        o[x][2 * r] *= f;
                        o[x][2 * r + 1] *= f;
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
            for (int x = 0; x < D / 16; ++x) {
                uint32_t vb[4];
                const int ch = 2 * x + vch;
                ldsm4_t(vt + (ch >> 3) * (kTile * 128) + vkey * 128 + (((ch ^ vkey) & 7) << 4), vb);
                mma16816(o[2 * x], pa, vb[0], vb[1]);
                mma16816(o[2 * x + 1], pa, vb[2], vb[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(smem_u32(&bars[C::kStages + s]));
        }
        // ---- the segment's end: join the eight warps in order, then o or the piece's (O, m, l) ----
        cons_sync();                                       // the last segment's ms, ls, red are read
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if ((lane & 3) == 0) {
                ms[warp][g + 8 * r] = m[r];
                ls[warp][g + 8 * r] = l[r];
            }
        }
        cons_sync();
        float f[2];
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            float M = -INFINITY;
#pragma unroll
            for (int x = 0; x < NW; ++x) M = fmaxf(M, ms[x][g + 8 * r]);
            f[r] = ex2(m[r] - (M == -INFINITY ? 0.f : M));
        }
        const bool whole = w.t0 == 0 && w.t1 == w.tiles;
        // slot 0: the piece's first segment
        float* part = a.part + ((int64_t)blockIdx.x * 2 + (w.left == u1 - u0 ? 0 : 1)) * kRows * (D + 2);
#pragma unroll
        for (int c = 0; c < D; c += CK) {
#pragma unroll
            for (int x = 0; x < CK / 8; ++x)
#pragma unroll
                for (int r = 0; r < HR; ++r)
                    *reinterpret_cast<float2*>(&red[warp][g + 8 * r][8 * x + q2]) =
                        make_float2(o[c / 8 + x][2 * r] * f[r], o[c / 8 + x][2 * r + 1] * f[r]);
            cons_sync();
            {
                // 256 threads x 2 columns = R8 x CK
                const int e = 2 * tid, r = e / CK, col = e % CK;
                float2 y = make_float2(0.f, 0.f);
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int x = 0; x < NW; ++x) {
                    const float2 z = *reinterpret_cast<const float2*>(&red[x][r][col]);
                    y.x += z.x;
                    y.y += z.y;
                    M = fmaxf(M, ms[x][r]);
                }
                const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int x = 0; x < NW; ++x) L = fmaf(ls[x][r], ex2(ms[x][r] - base), L);
                if (r < R) {
                    if (whole) {
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        T* O = reinterpret_cast<T*>(a.O.data) + (int64_t)w.b * a.O.row + (int64_t)(h0 + r) * a.O.head + c + col;
                        *reinterpret_cast<uint32_t*>(O) = pack2(y.x * inv, y.y * inv);
                        if (a.lse && c == 0 && col == 0)
                            a.lse[(int64_t)w.b * p.Hq + h0 + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * kAttnLn2;
                    } else {
                        *reinterpret_cast<float2*>(part + r * (D + 2) + c + col) = y;
                        if (c == 0 && col == 0) {
                            part[r * (D + 2) + D] = M;
                            part[r * (D + 2) + D + 1] = L;
                        }
                    }
                }
            }
            if (c + CK < D) cons_sync();
        }
    } while (w.next(p, a.I));
    if (!ok && lane == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
}

// Joins the pieces of one split item: CTA (c, r) takes row r of the item that begins in piece c
// and goes on behind it, if there is one.
template <typename T, int D>
__global__ void __launch_bounds__(512) paged_join_kernel(const Args a) {
    constexpr int NG = 512 / D;
    __shared__ int64_t scan[512 / kWarp];
    __shared__ float acc_sm[NG][D], l_sm[NG];
    __shared__ float red[512 / kWarp];
    const PagedArgs& p = a.p;
    const int c = blockIdx.x, r = blockIdx.y;
    auto count = [&](int b) -> int64_t { return (int64_t)tiles_of(p, b) * a.I; };
    const int64_t total = seq_total<512>(p.n_seq, count, scan);
    const int N = pieces_of(total);
    const int64_t u0 = c < N ? split_at(total, N, c) : 0, u1 = c < N ? split_at(total, N, c + 1) : 0;
    int b = 0;
    int64_t rem = 0;
    if (c < N) seq_find<512>(p.n_seq, count, u1 - 1, scan, &b, &rem);
    const int tiles = tiles_of(p, b), item = (int)(rem / tiles);
    const int64_t xs = u1 - 1 - rem % tiles, xe = xs + tiles;     // the item's units
    const int hk = item / a.RG, h0 = hk * p.G + (item % a.RG) * kRows;
    const int R = min(kRows, p.G - (item % a.RG) * kRows);
    // every CTA waits for the pieces: what comes behind this kernel relies on them being done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c >= N || xs < u0 || xe <= u1 || r >= R) return;
    const int c1 = split_of(total, N, xe - 1);
    const int np = c1 - c + 1;
    auto piece = [&](int i) {
        return a.part + ((int64_t)(c + i) * 2 + (i == 0 && xs != u0 ? 1 : 0)) * kRows * (D + 2) + r * (D + 2);
    };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < np; i += 512) m = fmaxf(m, piece(i)[D]);
    m = warp_max(m);
    if (threadIdx.x % kWarp == 0) red[threadIdx.x / kWarp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 512 / kWarp; ++i) m = fmaxf(m, red[i]);
    const float bs = m == -INFINITY ? 0.f : m;
    const int dim = threadIdx.x % D, g = threadIdx.x / D;
    float acc = 0.f, l = 0.f;
#pragma unroll 4
    for (int i = g; i < np; i += NG) {
        const float* q = piece(i);
        const float f = exp2f(q[D] - bs);
        acc = fmaf(f, q[dim], acc);
        l = fmaf(f, q[D + 1], l);
    }
    acc_sm[g][dim] = acc;
    if (dim == 0) l_sm[g] = l;
    __syncthreads();
    if (g == 0) {
        l = 0.f;
        acc = 0.f;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            l += l_sm[i];
            acc += acc_sm[i][dim];
        }
        const bool none = l == 0.f;
        IO<T>::st(reinterpret_cast<T*>(a.O.data), (int64_t)b * a.O.row + (int64_t)(h0 + r) * a.O.head + dim,
                  none ? 0.f : acc / l);
        if (a.lse && dim == 0)
            a.lse[(int64_t)b * p.Hq + h0 + r] = none ? -INFINITY : (m + log2f(l)) * kAttnLn2;
    }
}

Args make_args(const DecodeArgs& d) {
    Args a;
    a.p = d.p;
    a.Q = d.Q;
    a.O = d.O;
    a.lse = d.lse;
    a.part = d.part;
    a.scale_log2 = d.scale_log2;
    a.RG = (d.p.G + kRows - 1) / kRows;
    a.I = d.p.Hkv * a.RG;
    return a;
}

template <typename T, int D, typename K>
cudaError_t launch_kernel(K kernel, const DecodeArgs& d, cudaStream_t st) {
    using C = Cfg<T, D>;
    Maps maps;
    const auto ty = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t depth = (int64_t)d.p.n_pages * d.p.Hkv;
    const int rows = d.p.page < kTile ? d.p.page : kTile;
    if (!make_tmap3(&maps.k, ty, sizeof(T), d.p.K, D, d.p.page, depth, 128 / sizeof(T), rows) ||
        !make_tmap3(&maps.v, ty, sizeof(T), d.p.V, D, d.p.page, depth, 128 / sizeof(T), rows))
        return cudaErrorInvalidValue;
    const size_t smem = (size_t)C::kStages * 2 * C::kHalf + 1024;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<kPieces, kThreads, smem, st>>>(maps, make_args(d));
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_f32(const DecodeArgs& d, cudaStream_t st) {
    return d.p.G <= 4 ? launch_kernel<float, D>(paged_decode_kernel<float, D, 4>, d, st)
                      : launch_kernel<float, D>(paged_decode_kernel<float, D, kRows>, d, st);
}
template <int D>
cudaError_t launch_bf16(const DecodeArgs& d, cudaStream_t st) {
    return d.p.G <= 8 ? launch_kernel<__nv_bfloat16, D>(paged_decode_mma_kernel<D, true>, d, st)
                      : launch_kernel<__nv_bfloat16, D>(paged_decode_mma_kernel<D, false>, d, st);
}

template <typename T, int D>
cudaError_t launch_join(const DecodeArgs& d, cudaStream_t st) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(kPieces, d.p.G < kRows ? d.p.G : kRows);
    lc.blockDim = dim3(512);
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, paged_join_kernel<T, D>, make_args(d));
}

}  // namespace

int64_t paged_decode_workspace(int Hq, int Hkv, int d) { return (int64_t)kPieces * 2 * kRows * (d + 2) * sizeof(float); }

bool paged_decode_splits(const DecodeArgs& a) { return ((int64_t)a.p.width << a.p.page_log2) > kTile; }

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_f32<128>(a, st) : launch_f32<64>(a, st);
    return a.p.d == 128 ? launch_bf16<128>(a, st) : launch_bf16<64>(a, st);
}
cudaError_t launch_paged_join(const DecodeArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_join<float, 128>(a, st) : launch_join<float, 64>(a, st);
    return a.p.d == 128 ? launch_join<__nv_bfloat16, 128>(a, st) : launch_join<__nv_bfloat16, 64>(a, st);
}

cudaError_t paged_status_take(int32_t* bits, cudaStream_t st) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_status, sizeof(int32_t), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess || *bits == 0) return e;
    const int32_t zero = 0;
    e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

}  // namespace lola
