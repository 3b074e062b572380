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
constexpr float kRaise = 8.0f;            // bf16: m is set this far above a maximum (log2), and raised when one passes it
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
    int give_up;        // lola_selftest_attn_wait: a tile at which every third CTA gives up
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
    int given;       // segment slots given to the consumers, when the producer is done
    int arrived[2];  // this piece's record of that slot has been counted
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

// The segment [t0, t1) of an item of `tiles` tiles as one piece of it: the item's first unit is xs.
__device__ __forceinline__ void place_piece(const Start& st, int64_t xs, int tiles, Seg* g) {
    g->c0 = split_of(st.total, st.N, xs);
    g->np = split_of(st.total, st.N, xs + tiles - 1) - g->c0 + 1;
    g->k = (int)blockIdx.x - g->c0;
    g->s0 = xs != split_at(st.total, st.N, g->c0);
}

// The producer warp: segments and their tiles, in order.  A tile's pages outside the cache are not
// loaded; bit x of bad_sm marks the tile's x-th token box.  Segment i goes to slot i % NS.
template <typename T, int D, int NS, typename B>
__device__ __forceinline__ void produce(const Maps& maps, const Args& a, const Start& st, uint32_t ring, uint32_t qs,
                                        uint32_t q_pitch, B& bars, Seg* segs, uint32_t* bad_sm, int* abort_sm, int lane) {
    using C = Cfg<T, D>;
    const PagedArgs& p = a.p;
    const int box = min(p.page, kTile), lb = 31 - __clz(box), nbox = kTile >> lb;   // tokens of a box, boxes of a tile
    int b = st.b;
    int lens_b = b;                                               // the lanes hold 32 sequences' lengths
    int lens = b + lane < p.n_seq ? p.kv_len[b + lane] : 0;
    int64_t tokens = paged_tokens(p, __shfl_sync(0xffffffffu, lens, 0));
    int tiles = tiles_of(tokens), item = (int)(st.rem / tiles), t0 = (int)(st.rem % tiles);
    int64_t u = st.u0;
    int n = 0, i = 0, held_b = -1, held = -1;
    int held_c = 0;                                           // ... and 32 page-table columns of held_b
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
            if (!g.whole) place_piece(st, u - t0, tiles, &g);
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
        const bool give_up = gives_up(a.give_up, n, t1 - t0);
        const int stop = give_up ? t0 + a.give_up - n : t1;
        for (int t = t0; t < stop; ++t, ++n) {
            const int s = n % C::kStages;
            if (n >= C::kStages) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars.empty[s]), (uint32_t)(n / C::kStages - 1) & 1, abort_sm));
            if (!ok) break;
            // (positions fit 31 bits, but for the boxes behind the last token's)
            const uint32_t pos = (uint32_t)t * kTile, have = (uint32_t)tokens;
            const int col = (int)(pos >> p.page_log2);
            const int used = have > pos ? min(nbox, (int)((have - pos + box - 1) >> lb)) : 0;     // boxes with tokens
            if (held_b != b || col < held_c || col + used > held_c + 32) {
                held_b = b;
                held_c = col;
                const int64_t c = (int64_t)(col + lane) << p.page_log2;
                held = c < tokens ? paged_page(p, b, c) : 0;
            }
            // lanes 0 .. used - 1: a box of K each; lanes 16 ..: of V
            const int x = lane & 15;
            const int page = __shfl_sync(0xffffffffu, held, ((int)((pos + x * box) >> p.page_log2) - held_c) & 31);
            const bool mine = x < used, bad = mine && page < 0;
            const uint32_t bad_mask = __ballot_sync(0xffffffffu, bad) & 0xffffu;
            if (lane == 0) {
                if (bad_mask) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
                bad_sm[s] = bad_mask;
                mbar_expect(smem_u32(&bars.full[s]), (uint32_t)(2 * (used - __popc(bad_mask)) * box * C::kRowBytes));
                *reinterpret_cast<volatile int*>(&bars.issued) = n + 1;
            }
            __syncwarp();
            if (mine && !bad)
                tma_load4(ring + (uint32_t)s * 2 * C::kHalf + (lane >> 4) * C::kHalf + x * (uint32_t)(box * C::kRowBytes),
                          lane >> 4 ? &maps.v : &maps.k, 0, (int)((pos + x * box) & (p.page - 1)), 0, page * p.Hkv + hk,
                          smem_u32(&bars.full[s]));
        }
        if (give_up) {
            if (lane == 0) *reinterpret_cast<volatile int*>(abort_sm) = 1;
            ok = false;
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
    if (lane == 0) {
        if (!ok) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
        bars.given = i;
    }
}

// Whether sequence b has a token that can be seen (on a page of the cache).
__device__ __forceinline__ bool sees_token(const PagedArgs& p, int b) {
    const int64_t tokens = paged_tokens(p, p.kv_len[b]);
    for (int64_t pos = 0; pos < tokens; pos += p.page)
        if (paged_page(p, b, pos) >= 0) return true;
    return false;
}

// One row's 4 columns c .. c + 3: o, when all of the item's tokens are in, or a record
template <typename T, int D>
__device__ __forceinline__ void write_out(const Args& a, const Seg& g, bool whole, float* rec, int r, int c, float (&y)[4], float M, float L) {
    if (whole) {
        // (no token seen: o = 0; scores that are all minus infinity: 0 / 0)
        const float inv = L == 0.f ? (sees_token(a.p, g.b) ? NAN : 0.f) : 1.f / L;
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
// workspace needs no clearing, and a replayed graph, whose tag stays the same, finds no old count: every
// piece is counted, those of a CTA whose waits gave up too (settle).
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

// A join that piece k of an item takes part in: pieces c0 + step (first + x), x < cnt, the very first one's record
// in slot0.
struct Join {
    int k, np, step, slot0, slot;
    __device__ __forceinline__ explicit Join(const Seg& g) : k(g.k), np(g.np), step(1), slot0(g.s0), slot(0) {}
    __device__ __forceinline__ int first() const { return k / kJoin * kJoin; }
    __device__ __forceinline__ int cnt() const { return min(kJoin, np - first()); }
    __device__ __forceinline__ int head(const Seg& g) const { return g.c0 + step * first(); }
    __device__ __forceinline__ int hslot() const { return first() == 0 ? slot0 : slot; }
    // the second round: the joins, each in a record of its first piece
    __device__ __forceinline__ void next() {
        k /= kJoin;
        np = (np + kJoin - 1) / kJoin;
        step = kJoin;
        slot0 = 2 + slot0;
        slot = 2;
    }
};
// One more arrival; whether it is the last one of `cnt`.
template <int D>
__device__ __forceinline__ bool arrive(const Args& a, int head, int hslot, int cnt) {
    unsigned long long* c = cell<D>(a, head, hslot);
    unsigned long long old;
    asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(reinterpret_cast<uint64_t>(c)) : "memory");
    const bool last = (int)(old & 255) == cnt - 1;
    if (last) *reinterpret_cast<volatile unsigned long long*>(c) = 0ull;
    return last;
}

// Segment g's record is written by this group's NT threads (numbered t).  `bar` is their barrier.
template <typename T, int D, int NT, typename F>
__device__ void join_pieces(const Args& a, const Seg& g, int t, int* go, int* arrived, F&& bar) {
    for (Join join(g);; join.next()) {
        const int first = join.first(), cnt = join.cnt(), head = join.head(g), hslot = join.hslot(), slot = join.slot;
        const int np = join.np, step = join.step;
        bar();
        if (t == 0) {
            *go = arrive<D>(a, head, hslot, cnt);
            if (step == 1) arrived[g.k == 0 ? g.s0 : 0] = 1;
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
    }
}

// The end of a CTA whose waits gave up (all threads, after all roles): no copy is left in flight, and its pieces
// that were not counted are, so that every cell of the call ends at 0 (what the joins then make of their records
// is as invalid as the call).
template <int D, int S, int NS, typename B>
__device__ __noinline__ void settle(const Args& a, B& bars) {
    if (threadIdx.x == 0) {
        const int n = bars.issued, i = bars.given;
        for (int x = max(0, n - S); x < n; ++x) mbar_wait(smem_u32(&bars.full[x % S]), (uint32_t)(x / S) & 1, kWaitNs);
        for (int x = max(0, i - NS); x < i; ++x) mbar_wait(smem_u32(&bars.seg_full[x % NS]), (uint32_t)(x / NS) & 1, kWaitNs);
    }
    Start st;
    if (!find_start(a.p, a.I, &st) || threadIdx.x != 0) return;
    int b = st.b, tiles = tiles_of(paged_tokens(a.p, a.p.kv_len[b]));
    int item = (int)(st.rem / tiles), t0 = (int)(st.rem % tiles);
    for (int64_t u = st.u0; u < st.u1;) {
        const int t1 = (int)min((int64_t)tiles, t0 + (st.u1 - u));
        if (t0 > 0 || t1 < tiles) {
            Seg g;
            place_piece(st, u - t0, tiles, &g);
            if (!bars.arrived[g.k == 0 ? g.s0 : 0]) {
                open_cells<D>(a, g);
                for (Join join(g); arrive<D>(a, join.head(g), join.hslot(), join.cnt()) && join.cnt() < join.np;) join.next();
            }
        }
        u += t1 - t0;
        t0 = 0;
        if (++item == a.I && u < st.u1) {
            item = 0;
            tiles = tiles_of(paged_tokens(a.p, a.p.kv_len[++b]));
        }
    }
}

// ---- float32, CUDA cores ----
// Eight warps, the two halves of them on alternate tiles of a segment.  A warp takes four query rows and
// 64 / NP tokens of a tile (RM = 4, 8, 16 rows compiled for: NP = 4, 2, 1 parts of the tokens), 16 at a time,
// with its own running maximum, sum and output, joined at the segment's end: no barrier inside a segment (with
// all threads on one tile and two barriers in it, 64 sequences of 4000 tokens, 4 heads of 64, took 184 us, now 86).
// Lanes 8 tg + j: chunk j (16 bytes) of every 128-byte column of the rows, tokens 4 i + tg, so that K and V are
// read once, without bank conflicts, into products with q and the output in registers; the eight lanes' sums
// of a score are added and dealt out by halves (14 shuffles for 16 tokens x 4 rows).  m is the maximum so far:
// the largest weights' exponents stay near zero, where they lose least.
template <int D, int RM>
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
        bars.issued = bars.given = bars.arrived[0] = bars.arrived[1] = 0;
    }
    wait_for_last_kernel();
    Start st;
    if (!find_start(p, a.I, &st)) return;
    if (warp == NW) produce<float, D, 1>(maps, a, st, smem_u32(sm), smem_u32(Qs), D * 4, bars, segs, bad_sm, &abort_sm, lane);
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
        if (!g.whole && tid == 64) open_cells<D>(a, g);
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
            const int nk = max(0, min(kTile, g.len - t * kTile));
            const uint32_t bad = bad_sm[s];
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
        float* rec = record<D>(a, blockIdx.x, g.k == 0 ? g.s0 : 0);
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
            write_out<float, D>(a, g, g.whole, rec, r, c, y, M, ll);
        }
        if (!g.whole) join_pieces<float, D, kCons>(a, g, tid, &go, bars.arrived, bar);
        bar();                                                  // red, ms, ls are read
    }
    __syncthreads();
    if (abort_sm) settle<D, C::kStages, 1>(a, bars);
}

// ---- bf16: the tile products on the warps' matrix instructions ----
// Two groups of four warps: at d = 128 they take the segments in turn, so that one group's epilogue runs beside
// the other's tiles (64 sequences of 1000-8000 tokens, 32/8 heads, when both were built: 142 us, 152 on tiles in
// turn); at d = 64, where a tile's bytes come faster than four warps get through it, they take a segment's tiles in
// turn (64 x 8000 tokens, 16/8 heads, likewise: 171 us, 214 on segments in turn).  A warp takes 16 of a tile's 64 tokens, with its own running
// maximum, sum and output of the 16 query rows, joined at the segment's end.  S = Q K^T has the rows of Q as M, so
// that its accumulators are the A operand of P V as they stand.  m is raised lazily (it is set 8 above a
// maximum, so that no weight is above one), which leaves the output alone for most tiles.
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
        bars.issued = bars.given = bars.arrived[0] = bars.arrived[1] = 0;
    }
    wait_for_last_kernel();
    Start st;
    if (!find_start(p, a.I, &st)) return;
    if (warp == kCons / kWarp) produce<T, D, 2>(maps, a, st, sb, smem_u32(x.q[0]), M::kPitch, bars, segs, bad_sm, &abort_sm, lane);
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
        float* rec = record<D>(a, blockIdx.x, g.k == 0 ? g.s0 : 0);
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
                if (er < g.R) write_out<T, D>(a, g, g.whole, rec, er, c + ec, y, mm, ll);
            }
        }
        if (!g.whole) join_pieces<T, D, NT>(a, g, gt, &go[own], bars.arrived, bar);
    }
    __syncthreads();
    if (abort_sm) settle<D, C::kStages, 2>(a, bars);
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
    a.give_up = d.give_up;
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
    return launch_behind(kernel, kPieces, kThreads, smem, st, maps, make_args(d));
}
template <int D>
cudaError_t launch_f32(const DecodeArgs& d, cudaStream_t st) {
    static std::atomic<uint64_t> done[3] = {};
    if (d.p.G <= 4) return launch_kernel<float, D>(paged_decode_f32_kernel<D, 4>, done[0], d, st);
    if (d.p.G <= 8) return launch_kernel<float, D>(paged_decode_f32_kernel<D, 8>, done[1], d, st);
    return launch_kernel<float, D>(paged_decode_f32_kernel<D, 16>, done[2], d, st);
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

cudaError_t paged_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
