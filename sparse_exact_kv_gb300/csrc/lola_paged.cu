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
constexpr int kJoin = 16;                 // pieces joined at a time
constexpr uint64_t kWaitNs = 1000000000ull;

struct Maps {
    CUtensorMap k, v;   // [n_pages * Hkv][page][d] as 128-byte columns, boxes of min(page, 64) rows
};

struct Args {
    PagedArgs p;
    Rows Q, O;
    float* lse;
    float* part;        // workspace: records, then the joins' cells
    uint64_t tag;       // this call's mark in the cells (the low 8 bits are 0)
    float scale_log2;
    int RG, I;          // row groups per key/value head; items (row groups) per sequence
};

template <typename T, int D> struct Cfg {
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kHalf = kTile * kRowBytes;                // K or V of a tile
    static constexpr int kStages = 196608 / (2 * kHalf) > 12 ? 12 : 196608 / (2 * kHalf);
};

// ---- the workspace: per piece four records of (O [16][d], m [16], l [16]) -- its first segment's (slot
// 0), its last one's (1), and the joins of up to 16 pieces that begin with one of them (2, 3) -- and as
// many cells that count a join's arrivals ----
constexpr int kSlots = 4;
__host__ __device__ constexpr int64_t record_floats(int d) { return kRows * (int64_t)d + 2 * kRows; }
template <int D>
__device__ __forceinline__ float* record(const Args& a, int piece, int slot) {
    return a.part + ((int64_t)piece * kSlots + slot) * record_floats(D);
}
template <int D>
__device__ __forceinline__ unsigned long long* cell(const Args& a, int piece, int slot) {
    return reinterpret_cast<unsigned long long*>(a.part + (int64_t)kPieces * kSlots * record_floats(D)) + piece * kSlots + slot;
}

// Tiles of sequence b, for each of its items: at least one, so that an empty sequence's output
// is written too.
__device__ __forceinline__ int tiles_of(int64_t tokens) { return tokens <= 0 ? 1 : (int)((tokens + kTile - 1) / kTile); }

// Pieces of `total` units: none is empty.
__device__ __forceinline__ int pieces_of(int64_t total) { return (int)min((int64_t)kPieces, total); }

// One segment of the piece, published by the producer: `R` < 0 ends the consumers.
struct Seg {
    int b, h0, R;          // sequence, first query head, query rows
    int tiles, n0;         // tiles of the segment, number of its first one in the ring's order
    int len;               // tokens of the sequence from the segment's first tile on
    int whole;             // it covers the whole item
    int k, np, c0, s0;     // else: piece k of np, the first of them c0, whose record is slot s0
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store4(float* o, const float (&y)[4]) {
    *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* o, const float (&y)[4]) {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
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
// the producer has armed tile n's stage: only then does the parity of n's phase tell it from the one
// before (a group that has not waited for that one, which was another group's, would pass at once)
__device__ __forceinline__ bool issued_wait(const int* issued, int n, int* abort_sm) {
    if (*reinterpret_cast<const volatile int*>(issued) > n) return true;
    const uint64_t start = globaltimer_ns();
    while (*reinterpret_cast<const volatile int*>(issued) <= n) {
        if (*reinterpret_cast<volatile int*>(abort_sm)) return false;
        if (globaltimer_ns() - start > kWaitNs) {
            *abort_sm = 1;
            return false;
        }
    }
    return true;
}
// barrier `id` of a group of NT threads that also tells all of them whether one had x (so that a
// wait that gave up ends the whole group, and no barrier is left waiting)
template <int NT>
__device__ __forceinline__ bool group_or(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id), "n"(NT)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Barriers: a ring stage is full / empty; a segment slot (descriptor and Q rows) is full / empty.
template <int S> struct Bars {
    uint64_t full[S], empty[S], seg_full[2], seg_empty[2];
    int issued;      // tiles whose stage is armed
};

// Which piece this CTA is and where it begins (all threads): false if there is none.
struct Start {
    int64_t total, u0, u1, rem;   // units; rem: the first unit's number inside its sequence
    int N, b;
};
__device__ __forceinline__ bool find_start(const PagedArgs& p, int I, Start* st) {
    __shared__ int64_t sums[kThreads / kWarp];
    __shared__ int found_b;
    __shared__ int64_t found_r;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    auto count = [&](int b) -> int64_t { return b < p.n_seq ? (int64_t)tiles_of(paged_tokens(p, p.kv_len[b])) * I : 0; };
    const int64_t own = count(threadIdx.x);            // (the whole of it up to 288 sequences)
    int64_t rest = 0;
    for (int b = threadIdx.x + kThreads; b < p.n_seq; b += kThreads) rest += count(b);
    st->total = block_total<kThreads>(own + rest, sums);
    st->N = pieces_of(st->total);
    if ((int)blockIdx.x >= st->N) return false;
    st->u0 = split_at(st->total, st->N, blockIdx.x);
    st->u1 = split_at(st->total, st->N, blockIdx.x + 1);
    int64_t before = 0;
    for (int base = 0; base < p.n_seq; base += kThreads) {
        const int64_t x = base == 0 ? own : count(base + threadIdx.x);
        int64_t inc = x;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == kWarp - 1) sums[warp] = inc;
        __syncthreads();
        int64_t pre = before, all = before;
#pragma unroll
        for (int w = 0; w < kThreads / kWarp; ++w) {
            if (w < warp) pre += sums[w];
            all += sums[w];
        }
        const int64_t lo = pre + inc - x;
        if (st->u0 >= lo && st->u0 < lo + x) {
            found_b = base + threadIdx.x;
            found_r = st->u0 - lo;
        }
        if (st->u0 < all) break;
        before = all;
    }
    __syncthreads();
    st->b = found_b;
    st->rem = found_r;
    return true;
}

// The producer warp: segments and their tiles, in order.  A tile's pages outside the cache are not
// loaded; bit x of bad_sm marks the tile's x-th token box.  Segment i goes to slot i % NS.
template <typename T, int D, int NS, typename B>
__device__ __forceinline__ void produce(const Maps& maps, const Args& a, const Start& st, uint32_t ring, uint32_t qs,
                                        uint32_t q_pitch, B& bars, Seg* segs, uint32_t* bad_sm, int* abort_sm, int lane) {
    using C = Cfg<T, D>;
    const PagedArgs& p = a.p;
    const int box = min(p.page, kTile), nbox = kTile / box;       // tokens of a box, boxes of a tile
    int b = st.b;
    int lens_b = b;                                               // the lanes hold 32 sequences' lengths
    int lens = b + lane < p.n_seq ? p.kv_len[b + lane] : 0;
    int64_t tokens = paged_tokens(p, __shfl_sync(0xffffffffu, lens, 0));
    int tiles = tiles_of(tokens), item = (int)(st.rem / tiles), t0 = (int)(st.rem % tiles);
    int64_t u = st.u0;
    int n = 0, i = 0, held_b = -1, held = -1;
    int64_t held_c = 0;                                           // ... and 32 page-table columns of held_b
    bool ok = true;
    while (u < st.u1 && ok) {
        const int t1 = (int)min((int64_t)tiles, t0 + (st.u1 - u));
        const int hk = item / a.RG, h0 = hk * p.G + (item % a.RG) * kRows, R = min(kRows, p.G - (item % a.RG) * kRows);
        // ---- the segment's descriptor and Q rows ----
        const int slot = i % NS;
        if (i >= NS) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars.seg_empty[slot]), (uint32_t)(i / NS - 1) & 1, abort_sm));
        if (!ok) break;
        if (lane == 0) {
            Seg g;
            g.b = b;
            g.h0 = h0;
            g.R = R;
            g.tiles = t1 - t0;
            g.n0 = n;
            g.len = (int)max((int64_t)0, tokens - (int64_t)t0 * kTile);
            g.whole = t0 == 0 && t1 == tiles;
            g.k = g.np = g.c0 = g.s0 = 0;
            if (!g.whole) {
                const int64_t xs = u - t0;                        // the item's first unit
                g.c0 = split_of(st.total, st.N, xs);
                g.np = split_of(st.total, st.N, xs + tiles - 1) - g.c0 + 1;
                g.k = (int)blockIdx.x - g.c0;
                g.s0 = xs != split_at(st.total, st.N, g.c0);
            }
            segs[slot] = g;
            if (p.kv_len[b] > tokens && tokens > 0) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
            mbar_expect(smem_u32(&bars.seg_full[slot]), (uint32_t)(R * C::kRowBytes));
        }
        __syncwarp();
        if (lane < R)
            bulk_load(qs + (uint32_t)slot * kRows * q_pitch + lane * q_pitch,
                      a.Q.data + ((int64_t)b * a.Q.row + (int64_t)(h0 + lane) * a.Q.head) * (int)sizeof(T), C::kRowBytes,
                      smem_u32(&bars.seg_full[slot]));
        ++i;
        // ---- its tiles ----
        for (int t = t0; t < t1; ++t, ++n) {
            const int s = n % C::kStages;
            if (n >= C::kStages) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars.empty[s]), (uint32_t)(n / C::kStages - 1) & 1, abort_sm));
            if (!ok) break;
            const int64_t pos = (int64_t)t * kTile;
            const int64_t col = pos >> p.page_log2;
            const int used = (int)min((int64_t)nbox, (tokens - pos + box - 1) / box);       // boxes with tokens
            if (held_b != b || col < held_c || col + used > held_c + 32) {
                held_b = b;
                held_c = col;
                const int64_t c = (col + lane) << p.page_log2;
                held = c < tokens ? paged_page(p, b, c) : 0;
            }
            // lanes 0 .. used - 1: a box of K each; lanes 16 ..: of V
            const int x = lane & 15;
            const int page = __shfl_sync(0xffffffffu, held, (int)(((pos + x * box) >> p.page_log2) - held_c) & 31);
            const bool mine = x < used, bad = mine && page < 0;
            const uint32_t bad_mask = __ballot_sync(0xffffffffu, bad) & 0xffffu;
            if (lane == 0) {
                if (bad_mask) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
                bad_sm[s] = bad_mask;
                mbar_expect(smem_u32(&bars.full[s]), (uint32_t)(2 * (max(used, 0) - __popc(bad_mask)) * box * C::kRowBytes));
                *reinterpret_cast<volatile int*>(&bars.issued) = n + 1;
            }
            __syncwarp();
            if (mine && !bad)
                tma_load4(ring + (uint32_t)s * 2 * C::kHalf + (lane >> 4) * C::kHalf + x * (uint32_t)(box * C::kRowBytes),
                          lane >> 4 ? &maps.v : &maps.k, 0, (int)((pos + x * box) & (p.page - 1)), 0, page * p.Hkv + hk,
                          smem_u32(&bars.full[s]));
        }
        u += t1 - t0;
        t0 = 0;
        if (++item == a.I && u < st.u1) {
            item = 0;
            ++b;
            if (b >= lens_b + 32) {
                lens_b = b;
                lens = b + lane < p.n_seq ? p.kv_len[b + lane] : 0;
            }
            tokens = paged_tokens(p, __shfl_sync(0xffffffffu, lens, b - lens_b));
            tiles = tiles_of(tokens);
        }
    }
    // the consumers' end
    for (int e = 0; e < NS && ok; ++e, ++i) {
        const int slot = i % NS;
        if (i >= NS) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars.seg_empty[slot]), (uint32_t)(i / NS - 1) & 1, abort_sm));
        if (ok && lane == 0) {
            segs[slot].R = -1;
            mbar_arrive1(smem_u32(&bars.seg_full[slot]));
        }
    }
    // leave no copy in flight
    if (!ok && lane == 0) {
        atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
        for (int x = max(0, n - C::kStages); x < n; ++x) mbar_wait(smem_u32(&bars.full[x % C::kStages]), (uint32_t)(x / C::kStages) & 1, kWaitNs);
        for (int x = max(0, i - NS); x < i; ++x) mbar_wait(smem_u32(&bars.seg_full[x % NS]), (uint32_t)(x / NS) & 1, kWaitNs);
    }
}

// One row's 4 columns c .. c + 3: o, when all of the item's tokens are in, or a record
template <typename T, int D>
__device__ __forceinline__ void write_out(const Args& a, const Seg& g, bool whole, float* rec, int r, int c, float (&y)[4], float M, float L) {
    if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;            // (no token seen: o = 0)
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] *= inv;
        store4(reinterpret_cast<T*>(a.O.data) + (int64_t)g.b * a.O.row + (int64_t)(g.h0 + r) * a.O.head + c, y);
        if (a.lse && c == 0) a.lse[(int64_t)g.b * a.p.Hq + g.h0 + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * kAttnLn2;
    } else {
        store4(rec + r * D + c, y);
        if (c == 0) {
            rec[kRows * D + r] = M;
            rec[kRows * D + kRows + r] = L;
        }
    }
}

// ---- the join of an item's pieces ----
// Up to 16 pieces are joined at once, by the last of them to arrive; an item of more pieces takes a
// second round over those joins.  A join counts its arrivals in a cell that holds the call's tag (56
// bits) and the count (8): whoever takes part first swaps whatever the workspace held for the tag and a
// count of 0 -- long before its own arrival, off the critical path -- and the last one leaves 0.  So a
// workspace needs no clearing, and a replayed graph, whose tag stays the same, finds no old count.
template <int D>
__device__ __forceinline__ void open_cell(const Args& a, int piece, int slot) {
    unsigned long long* c = cell<D>(a, piece, slot);
    const unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(c);
    if ((old ^ a.tag) >> 8) atomicCAS(c, old, (unsigned long long)a.tag);   // (a failure: another one was faster)
}
template <int D>
__device__ __forceinline__ void open_cells(const Args& a, const Seg& g) {
    const int first = g.k / kJoin * kJoin;
    open_cell<D>(a, g.c0 + first, first == 0 ? g.s0 : 0);
    if (g.np > kJoin) open_cell<D>(a, g.c0, 2 + g.s0);
}

// Segment g's record is written by this group's NT threads (numbered t).  `bar` is their barrier.
template <typename T, int D, int NT, typename F>
__device__ void join_pieces(const Args& a, const Seg& g, int t, int* go, F&& bar) {
    int k = g.k, np = g.np, step = 1, slot0 = g.s0, slot = 0;
    for (;;) {
        // members of this join: pieces c0 + step (first + x), x < cnt, the very first one's record in slot0
        const int first = k / kJoin * kJoin, cnt = min(kJoin, np - first);
        const int head = g.c0 + step * first, hslot = first == 0 ? slot0 : slot;
        bar();
        if (t == 0) {
            unsigned long long old;
            asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;"
                         : "=l"(old)
                         : "l"(reinterpret_cast<uint64_t>(cell<D>(a, head, hslot)))
                         : "memory");
            const bool last = (int)(old & 255) == cnt - 1;
            if (last) *reinterpret_cast<volatile unsigned long long*>(cell<D>(a, head, hslot)) = 0ull;
            *go = last;
        }
        bar();
        if (!*go) return;
        const float* rec0 = record<D>(a, head, hslot);
        const int64_t stride = (int64_t)step * kSlots * record_floats(D);    // from a member's record to the next
        const int64_t shift = (int64_t)(slot - hslot) * record_floats(D);    // (the first may sit in another slot)
        for (int e = t; e < g.R * (D / 4); e += NT) {
            const int r = e / (D / 4), c = e % (D / 4) * 4;
            float m[kJoin], l[kJoin];
            float4 z[kJoin];
#pragma unroll
            for (int x = 0; x < kJoin; ++x) {
                const float* rec = rec0 + x * stride + (x > 0 ? shift : 0);
                m[x] = x < cnt ? __ldcg(rec + kRows * D + r) : -INFINITY;
                l[x] = x < cnt ? __ldcg(rec + kRows * D + kRows + r) : 0.f;
                z[x] = x < cnt ? __ldcg(reinterpret_cast<const float4*>(rec + r * D + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float M = -INFINITY, L = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < kJoin; ++x) M = fmaxf(M, m[x]);
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int x = 0; x < kJoin; ++x) {
                const float f = ex2(m[x] - base);
                L = fmaf(f, l[x], L);
                y[0] = fmaf(f, z[x].x, y[0]);
                y[1] = fmaf(f, z[x].y, y[1]);
                y[2] = fmaf(f, z[x].z, y[2]);
                y[3] = fmaf(f, z[x].w, y[3]);
            }
            write_out<T, D>(a, g, cnt == np, record<D>(a, head, 2 + hslot), r, c, y, M, L);
        }
        if (cnt == np) return;
        // the second round: the joins, each in a record of its first piece
        k /= kJoin;
        np = (np + kJoin - 1) / kJoin;
        step = kJoin;
        slot0 = 2 + slot0;
        slot = 2;
    }
}

// ---- float32, CUDA cores: 256 threads take a tile together ----
// Scores: a thread has one token and every fourth row; P V: a thread has one channel of every row over
// its share of the tokens.  RM: rows compiled for (4 or 16).
template <int D, int RM>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_f32_kernel(const __grid_constant__ Maps maps, const Args a) {
    using C = Cfg<float, D>;
    constexpr int KP = kCons / D, NW = kCons / kWarp;           // key parts of P V
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) Bars<C::kStages> bars;
    __shared__ uint32_t bad_sm[C::kStages];
    __shared__ int abort_sm, go;
    __shared__ Seg segs[1];
    __shared__ __align__(16) float Qs[kRows][D];
    // the weights of two tiles, and at a segment's end its outputs by key part
    __shared__ __align__(16) float shared_sr[KP * RM * D > 2 * RM * kTile ? KP * RM * D : 2 * RM * kTile];
    auto Ss = reinterpret_cast<float(*)[RM][kTile]>(shared_sr);
    auto red = reinterpret_cast<float(*)[RM][D]>(shared_sr);
    __shared__ float fs[2][RM], ms[kRows], ls[kRows];
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 1);
            mbar_init(smem_u32(&bars.empty[s]), NW);
        }
        mbar_init(smem_u32(&bars.seg_full[0]), 1);
        mbar_init(smem_u32(&bars.seg_empty[0]), NW);
        abort_sm = 0;
        bars.issued = 0;
    }
    Start st;
    if (!find_start(p, a.I, &st)) return;
    if (warp == NW) {
        produce<float, D, 1>(maps, a, st, smem_u32(sm), smem_u32(Qs), D * 4, bars, segs, bad_sm, &abort_sm, lane);
        return;
    }
    auto bar = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    const int key = tid % kTile, hs = tid / kTile;
    const int dim = tid % D, part = tid / D;
    const int box = min(p.page, kTile), lb = 31 - __clz(box);
    // byte offset of 16-byte chunk 0 of a token's row; column x (128 bytes) is x * box * 128 further
    auto row_at = [&](int k) { return (k >> lb) * box * C::kRowBytes + (k & (box - 1)) * 128; };
    for (int i = 0;; ++i) {
        if (group_or<kCons>(1, !ring_wait(smem_u32(&bars.seg_full[0]), (uint32_t)i & 1, &abort_sm))) {
            if (tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
        const Seg g = segs[0];
        if (g.R < 0) break;
        if (!g.whole && tid == 64) open_cells<D>(a, g);
        if (tid < RM) {
            ms[tid] = -INFINITY;
            ls[tid] = 0.f;
        }
        float acc[RM];
#pragma unroll
        for (int r = 0; r < RM; ++r) acc[r] = 0.f;
        bar();
        bool ok = true;
        for (int t = 0; t < g.tiles; ++t) {
            const int n = g.n0 + t, s = n % C::kStages, e = n & 1;
            ok = ok && ring_wait(smem_u32(&bars.full[s]), (uint32_t)(n / C::kStages) & 1, &abort_sm);
            const uint8_t* Kt = sm + (size_t)s * 2 * C::kHalf;
            const uint8_t* Vt = Kt + C::kHalf;
            const int nk = max(0, min(kTile, g.len - t * kTile));
            const uint32_t bad = ok ? bad_sm[s] : ~0u;
            float sc[(RM + 3) / 4];
#pragma unroll
            for (int x = 0; x < (RM + 3) / 4; ++x) sc[x] = 0.f;
            const bool seen = key < nk && !((bad >> (key >> lb)) & 1u);
            const uint8_t* kr = Kt + row_at(key);
#pragma unroll 4
            for (int c = 0; c < D / 4; ++c) {
                const float4 kv = *reinterpret_cast<const float4*>(kr + (c >> 3) * (box * 128) + (((c ^ key) & 7) << 4));
#pragma unroll
                for (int x = 0; x < (RM + 3) / 4; ++x) {
                    const float4 q = *reinterpret_cast<const float4*>(&Qs[hs + 4 * x][4 * c]);
                    sc[x] = fmaf(q.x, kv.x, sc[x]);
                    sc[x] = fmaf(q.y, kv.y, sc[x]);
                    sc[x] = fmaf(q.z, kv.z, sc[x]);
                    sc[x] = fmaf(q.w, kv.w, sc[x]);
                }
            }
#pragma unroll
            for (int x = 0; x < (RM + 3) / 4; ++x) Ss[e][hs + 4 * x][key] = seen ? sc[x] * a.scale_log2 : -INFINITY;
            bar();
            // running maximum and sum: warp w takes rows w, w + 8
            for (int r = warp; r < RM; r += NW) {
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
            bar();
#pragma unroll
            for (int r = 0; r < RM; ++r) acc[r] *= fs[e][r];
            constexpr int KN = kTile / KP;
            const int ch = dim / 4;
            const uint8_t* vb = Vt + (ch >> 3) * (box * 128) + (dim & 3) * 4;
            for (int k4 = part * KN; k4 < min(nk, (part + 1) * KN); k4 += 4) {
                float v[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int kk = k4 + x;
                    // (a token that is not seen has p = 0; its value row may be anything)
                    const bool in = kk < nk && !((bad >> (kk >> lb)) & 1u);
                    v[x] = in ? *reinterpret_cast<const float*>(vb + row_at(kk) + (((ch ^ kk) & 7) << 4)) : 0.f;
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
            if (lane == 0) mbar_arrive1(smem_u32(&bars.empty[s]));
        }
        // ---- the segment's end: add the key parts in order ----
        if (group_or<kCons>(1, !ok)) {
            if (tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
#pragma unroll
        for (int r = 0; r < RM; ++r) red[part][r][dim] = acc[r];
        bar();
        float* rec = record<D>(a, blockIdx.x, g.k == 0 ? g.s0 : 0);
        for (int e = tid; e < g.R * (D / 4); e += kCons) {
            const int r = e / (D / 4), c = e % (D / 4) * 4;
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int z = 0; z < 4; ++z) y[z] += red[k][r][c + z];
            write_out<float, D>(a, g, g.whole, rec, r, c, y, ms[r], ls[r]);
        }
        if (!g.whole) join_pieces<float, D, kCons>(a, g, tid, &go, bar);
        bar();                                                  // Qs, red, ms, ls are read
        if (lane == 0) mbar_arrive1(smem_u32(&bars.seg_empty[0]));
    }
}

// ---- bf16: the tile products on the warps' matrix instructions ----
// Two groups of four warps take the segments in turn, so that one group's epilogue runs beside the
// other's tiles; a warp takes 16 of a tile's 64 tokens, with its own running maximum, sum and
// output of the 16 query rows, joined at the segment's end.  S = Q K^T has the rows of Q as M, so
// that its accumulators are the A operand of P V as they stand.  m is raised lazily (by more than
// 2^8 at a time), which leaves the output alone for most tiles.
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
constexpr float kRaise = 8.0f;

template <int D, bool HALF> struct MmaSmem {
    static constexpr int HR = HALF ? 1 : 2, R8 = 8 * HR, CK = 512 / R8;     // rows kept; columns joined at a time
    static constexpr int kPitch = 2 * D + 16;                               // Q rows (16-byte shift against bank conflicts)
    float red[2][4][R8][CK];
    float ms[2][4][R8], ls[2][4][R8];
    uint8_t q[2][kRows * kPitch];
};

// HALF: at most 8 query rows (rows 8-15 of the products hold anything and are left alone)
template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_mma_kernel(const __grid_constant__ Maps maps, const Args a) {
    using T = __nv_bfloat16;
    using C = Cfg<T, D>;
    using M = MmaSmem<D, HALF>;
    constexpr int HR = M::HR, CK = M::CK;
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
            mbar_init(smem_u32(&bars.seg_empty[s]), 4);
        }
        abort_sm = 0;
        bars.issued = 0;
    }
    Start st;
    if (!find_start(p, a.I, &st)) return;
    if (warp == kCons / kWarp) {
        produce<T, D, 2>(maps, a, st, sb, smem_u32(x.q[0]), M::kPitch, bars, segs, bad_sm, &abort_sm, lane);
        return;
    }
    const int grp = warp >> 2, wg = warp & 3, gt = tid & 127, g8 = lane >> 2, q2 = (lane & 3) * 2;
    auto bar = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory"); };
    const int k0 = wg * 16;                                            // this warp's tokens of a tile
    const int box = min(p.page, kTile), lb = 31 - __clz(box);
    const uint32_t col = (uint32_t)box * 128;                          // from one 128-byte column to the next
    auto row_at = [&](int k) { return (uint32_t)((k >> lb) * box * C::kRowBytes + (k & (box - 1)) * 128); };
    const int kkey = k0 + ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;        // ldmatrix rows of K
    const int vkey = k0 + (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;        // ... of V
    const uint32_t krow = row_at(kkey), vrow = C::kHalf + row_at(vkey);
    const uint32_t qrow = smem_u32(x.q[grp]) + ((lane & 7) + ((lane >> 3) & 1) * 8) * M::kPitch + (lane >> 4) * 16;
    for (int i = 0;; ++i) {
        if (group_or<128>(1 + grp, !ring_wait(smem_u32(&bars.seg_full[grp]), (uint32_t)i & 1, &abort_sm))) {
            if (gt == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
        const Seg g = segs[grp];
        if (g.R < 0) break;
        if (!g.whole && gt == 64) open_cells<D>(a, g);
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int y = 0; y < D / 16; ++y) ldsm4(qrow + 32 * y, qa[y]);
        __syncwarp();
        if (lane == 0) mbar_arrive1(smem_u32(&bars.seg_empty[grp]));   // (g and the Q rows are in registers)
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[y][e] = 0.f;
        bool ok = true;
        for (int t = 0; t < g.tiles; ++t) {
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
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2)) * a.scale_log2;
                const bool need = bm > m[r] + kRaise || (m[r] == -INFINITY && bm > m[r]);
                if (__any_sync(0xffffffffu, need)) {
                    const float f = need ? ex2(m[r] - bm) : 1.f;
                    if (need) m[r] = bm;
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
        // ---- the segment's end: add the four warps in order, then o or the piece's record ----
        if (group_or<128>(1 + grp, !ok)) {
            if (gt == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if ((lane & 3) == 0) {
                x.ms[grp][wg][g8 + 8 * r] = m[r];
                x.ls[grp][wg][g8 + 8 * r] = l[r];
            }
        }
        bar();
        float f[2];
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) mm = fmaxf(mm, x.ms[grp][w][g8 + 8 * r]);
            f[r] = ex2(m[r] - (mm == -INFINITY ? 0.f : mm));
        }
        float* rec = record<D>(a, blockIdx.x, g.k == 0 ? g.s0 : 0);
        const int er = 4 * gt / CK, ec = 4 * gt % CK;          // 128 threads x 4 columns = R8 x CK
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) mm = fmaxf(mm, x.ms[grp][w][er]);
#pragma unroll
        for (int w = 0; w < 4; ++w) ll = fmaf(x.ls[grp][w][er], ex2(x.ms[grp][w][er] - (mm == -INFINITY ? 0.f : mm)), ll);
#pragma unroll
        for (int c = 0; c < D; c += CK) {
            if (c > 0) bar();
#pragma unroll
            for (int y = 0; y < CK / 8; ++y)
#pragma unroll
                for (int r = 0; r < HR; ++r)
                    *reinterpret_cast<float2*>(&x.red[grp][wg][g8 + 8 * r][8 * y + q2]) =
                        make_float2(o[c / 8 + y][2 * r] * f[r], o[c / 8 + y][2 * r + 1] * f[r]);
            bar();
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 z = *reinterpret_cast<const float4*>(&x.red[grp][w][er][ec]);
                y[0] += z.x;
                y[1] += z.y;
                y[2] += z.z;
                y[3] += z.w;
            }
            if (er < g.R) write_out<T, D>(a, g, g.whole, rec, er, c + ec, y, mm, ll);
        }
        if (!g.whole) join_pieces<T, D, 128>(a, g, gt, &go[grp], bar);
    }
}

Args make_args(const DecodeArgs& d) {
    Args a;
    a.p = d.p;
    a.Q = d.Q;
    a.O = d.O;
    a.lse = d.lse;
    a.part = d.part;
    a.tag = d.tag << 8;
    a.scale_log2 = d.scale_log2;
    a.RG = (d.p.G + kRows - 1) / kRows;
    a.I = d.p.Hkv * a.RG;
    return a;
}

template <typename T, int D, typename K>
cudaError_t launch_kernel(K kernel, std::atomic<uint64_t>& done, const DecodeArgs& d, cudaStream_t st) {
    using C = Cfg<T, D>;
    Maps maps;
    const auto ty = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t depth = (int64_t)d.p.n_pages * d.p.Hkv;
    const int rows = d.p.page < kTile ? d.p.page : kTile;
    if (!make_tmap_pages(&maps.k, ty, sizeof(T), d.p.K, D, d.p.page, depth, rows, D * (int)sizeof(T) / 128) ||
        !make_tmap_pages(&maps.v, ty, sizeof(T), d.p.V, D, d.p.page, depth, rows, D * (int)sizeof(T) / 128))
        return cudaErrorInvalidValue;
    const size_t smem = (size_t)C::kStages * 2 * C::kHalf + 1024;
    cudaError_t e = opt_in_smem(kernel, (int)smem, done);
    if (e != cudaSuccess) return e;
    kernel<<<kPieces, kThreads, smem, st>>>(maps, make_args(d));
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_f32(const DecodeArgs& d, cudaStream_t st) {
    static std::atomic<uint64_t> done[2] = {};
    return d.p.G <= 4 ? launch_kernel<float, D>(paged_decode_f32_kernel<D, 4>, done[0], d, st)
                      : launch_kernel<float, D>(paged_decode_f32_kernel<D, kRows>, done[1], d, st);
}
template <int D>
cudaError_t launch_bf16(const DecodeArgs& d, cudaStream_t st) {
    static std::atomic<uint64_t> done[2] = {};
    return d.p.G <= 8 ? launch_kernel<__nv_bfloat16, D>(paged_decode_mma_kernel<D, true>, done[0], d, st)
                      : launch_kernel<__nv_bfloat16, D>(paged_decode_mma_kernel<D, false>, done[1], d, st);
}

}  // namespace

int64_t paged_decode_workspace(int d) { return (int64_t)kPieces * kSlots * (record_floats(d) * sizeof(float) + sizeof(uint64_t)); }

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_f32<128>(a, st) : launch_f32<64>(a, st);
    return a.p.d == 128 ? launch_bf16<128>(a, st) : launch_bf16<64>(a, st);
}

cudaError_t paged_status_take(int32_t* bits, cudaStream_t st) { return take_word(g_status, bits, st); }

}  // namespace lola
