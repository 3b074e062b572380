// K12: attention of many sequences' query tokens over the prefixes that they share (bfloat16 io, tensor cores).
//
// The rows of a prefix and key head are the query heads of all sequences that share it: up to 256 of them are an item,
// two tiles of 128 (MMA M = 128, TMEM lane = row), which read every block of 128 keys once:
//   S = Q K^T,  P = 2^{c S - m},  l += sum P,  O += P V.
// No row is masked but by the prefix' length.  The (prefix, key head, 256 rows, block) units are counted in that order
// and cut into as many equal pieces as there are SMs, so that one prefix alone fills the GPU; a piece leaves (m, l, O) of
// each of its segments for the kernel that joins them (lola_shared.cu).  With one prefix of more than 256 rows, the row
// items of the same keys are side by side in time: the units are (key head, block), and as many CTAs as there are row
// items take a piece, so that keys and values come from HBM once (counted one item behind the other, 512 rows of
// 128000 tokens read them twice: 8 heads, d = 128, 218 us).
// An item of up to 128 rows has one tile of them: then its two halves are the even and the odd blocks, so that one half's
// softmax runs beside the other's products, and the halves are added at the segment's end.
// Warps: 0-3, 4-7 softmax of tile 0, 1 (one thread per row: Q rows to shared memory, S into registers, maximum, weights, P
// into TMEM over S, at the end O out of TMEM); 8 products (one thread); 9 pages and loads, a ring of K and V blocks.
// QZ, a quantised cache: the ring's blocks are written by warps 12-15 (or, by turns, 12-15 and 16-19), as float16 numbers,
// from e4m3 numbers and powers of two that a second ring brings.  Where the powers of a block's keys, or of its values, lie
// close together (kApart), the numbers are code 2^(e - E), E the largest of them, exactly; a key's 2^E is a factor of the
// block's scores, a value's joins the weights' exponent.  Else they are the codes as they stand, and the softmax takes every
// token's powers out of a table in shared memory: score by score, a branch that blocks of the other kind pass by.  So no row
// costs others their bits, whatever its power and its weight.  The rows of Q with powers of two of their own, the weights
// times 2^15, and l in the scores' unit, apart from the weights', are lola_quant.cu's.
// (Blocks of bfloat16 numbers code 2^e, by shifts, two products a pair and a look for NaN, took the four warps 3.4 us for
// K and V.)
// m is raised lazily, as in lola_attn_tc.cu: it is set 8 above a maximum, so that no weight is above one.
// Long prefixes: bfloat16, 128 sequences behind 131072 tokens, 32/8 heads, d = 128, 198 us, 1390 TFLOP/s, bound by the way from
// scores to weights beside the products; a quantised cache 259 us, 1060 TFLOP/s, bound by the conversion beside that (a block
// of K or V takes its four warps 560 clocks alone, 1300 there).  Short ones by their start: 64 sequences behind 16001
// tokens take 33 us, of which lookups, TMEM and the first block are 6 and the first pass through the softmax's code, which
// comes into the instruction caches meanwhile, another 5 (a pass over an empty block ahead of the first one, less code, and
// fewer loads at the start were each built and measured: no gain).
// Every wait is bounded (1 s, then LOLA_ATTN_TIMEOUT).
#include "lola_attn_mma.cuh"
#include "lola_codes.cuh"
#include "lola_paged.cuh"

namespace lola {
namespace {

constexpr int kM = 128;                  // rows of a tile
constexpr int kN = 128;                  // keys of a block
constexpr int kItem = kPrefixRows;       // rows of an item: two tiles
static_assert(kItem == 2 * kM, "two tiles");
constexpr int kBad = 8;                  // blocks whose pages and powers are remembered: more than the loader is ahead
// QZ: how far a block's powers lie apart at most to enter its numbers.  Keys: code 2^-15 is still a multiple of 2^-24, which
// float16 has.  Values: m is set above a block's largest score and largest power, which may be different tokens'; the
// largest weight is then 2^-16 at least, 2^-8 for that and 2^-8 for m's own distance, and weights keep their 11 bits down
// to 2^-13 of it (2^-29, below which float16 numbers of 2^15 w have fewer).
constexpr int kApartKeys = 15, kApartValues = 8;
// Blocks whose tokens' powers are kept, converted and not yet weighed: without block j's weights its V stays in the ring, and
// the conversion comes kRing - 1 stages, two key blocks (two tiles) or three (one: V of j is stage 2 j + 2), further.
constexpr int kTables = 4;
constexpr int kTableBytes = 2 * kN;

// CV: groups of four converting warps.
template <int D, bool QZ, int CV> struct PCfg {
    static constexpr int kThreads = 384 + 128 * CV;
    static constexpr int kMmaWarp = 8, kLoadWarp = 9, kConvWarp = 12;
    static constexpr int kTileBytes = kM * D * 2;                       // a Q tile, a K or V block
    static constexpr int kRing = D == 128 ? (QZ ? 3 : 5) : (QZ ? 4 : 8);
    static constexpr int kRaw = QZ ? (D == 128 ? 4 : 8) : 1;            // blocks of codes (K or V)
    static constexpr int kRawBytes = QZ ? kN * D + 2 * kN : 0;         // codes, their powers, behind keys the values' powers too
    // (behind that: QZ the tables, else what aligning takes)
    static constexpr int kTableAt = (2 + kRing) * kTileBytes + kRaw * kRawBytes;
    static constexpr int kSmem = kTableAt + 1024;
    static_assert(kTables * kTableBytes <= 1024, "tables");
    // Registers of a softmax thread and of the others: what the block was launched with, 168, 128 or 96 a thread, given out
    // anew, so that a row's 128 scores fit.  QZ at d = 64: the scores come first here too (64 sequences behind 64000 tokens,
    // 32/8 heads: 60 us, 68 with 128 and 128).
    static constexpr int kSoftmaxRegs = QZ ? (D == 128 ? 128 : 192) : 208, kOtherRegs = QZ ? (D == 64 ? 64 : CV == 2 ? 72 : 128) : 88;
    static constexpr int kLaunchRegs = QZ ? (CV == 2 ? 96 : 128) : 168;
    static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs, "more than the block has");
    // Scores in registers.  QZ at d = 128 is bound by the conversion, whose warps need their 128 registers and the schedulers'
    // time: the softmax goes over S twice there, 32 columns at a time (128 sequences behind 131072 tokens, 32/8 heads: 256 us,
    // half of the scores held 300, all of them, with 192 and 64 registers, 334).  Elsewhere S is
    // read once (bfloat16, the same size: 198 us, 221 in the loop; QZ, d = 64, 24/4 heads: 162 and 171).
    static constexpr int kHeld = QZ && D == 128 ? 32 : kN;
    __device__ static constexpr uint32_t TS(int i) { return 128u * i; }  // S (P over its first half)
    __device__ static constexpr uint32_t TO(int i) { return 256u + (uint32_t)D * i; }
};

// A segment: blocks of one item.  nb < 0: there are no more.
struct PSeg {
    int m0, r0, R, hk;         // first sequence of the prefix; first row of the item among the prefix' rows, rows
    int nb, len;               // blocks; tokens from the first one on
    int n0, blk0;              // numbers of the first stage and block, over all segments
    int whole, k, np, rec;     // as in Seg; rec: the item's first record
};

// Which of columns x0 .. x0 + 31 of a block are tokens that are seen.
__device__ __forceinline__ uint32_t seen_columns(int x0, int valid, uint32_t bad, int lb) {
    uint32_t seen = valid >= x0 + 32 ? ~0u : valid <= x0 ? 0u : (1u << (valid - x0)) - 1u;
    for (int x = 0; x < 32; x += 1 << min(lb, 5))
        if ((bad >> ((x0 + x) >> lb)) & 1u) seen &= lb >= 5 ? 0u : ~(((1u << (1 << lb)) - 1u) << x);
    return seen;
}

// The row's outputs, `width` columns from `to` on, times f.
__device__ __forceinline__ void scale_output(uint32_t to, int width, float f) {
#pragma unroll 1
    for (int x = 0; x < width; x += 16) {
        uint32_t o[16];
        tmem_ld16(to + x, o);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
        tmem_st16(to + x, o);
    }
}
// QZ, a block whose powers lie too far apart: a row's softmax score by score, m, l and ml before and after it in x.  (A call,
// so that these blocks' code costs the others no registers.)
struct ByToken {
    uint32_t ts, to, table, bad;  // TMEM: S, O; shared memory: 128 powers of the keys, 128 of the values (biased)
    float c;
    int valid, lb, width;
};
__device__ __forceinline__ uint32_t table_word(uint32_t at) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at));
    return w;
}
// columns x0 .. x0 + 31: scores, minus infinity for tokens that are not seen; and the values' powers, which their weights'
// exponents have besides
__device__ __forceinline__ void token_scores(const ByToken& t, int x0, float (&s)[32]) {
    tmem_ld32(t.ts + x0, s);
    tmem_wait_ld();
    const uint32_t seen = seen_columns(x0, t.valid, t.bad, t.lb);
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
        const uint32_t w = table_word(t.table + x0 + x);
#pragma unroll
        for (int y = 0; y < 4; ++y)
            s[x + y] = (seen >> (x + y)) & 1u ? s[x + y] * t.c * __uint_as_float(((w >> (8 * y)) & 255u) << 23) : -INFINITY;
    }
}
__device__ __forceinline__ void token_powers(const ByToken& t, int x0, float (&s)[32]) {
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
        const uint32_t w = table_word(t.table + kN + x0 + x);
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x + y] += (float)(int)((w >> (8 * y)) & 255u) - 127.f;
    }
}
__device__ __noinline__ float3 by_token_block(const ByToken t, bool first, float3 x) {
    float m = x.x, l = x.y, high = x.z, top = -INFINITY;
#pragma unroll 1
    for (int x0 = 0; x0 < kN; x0 += 32) {
        float s[32], now = high;
        token_scores(t, x0, s);
#pragma unroll
        for (int y = 0; y < 32; ++y) now = fmaxf(now, s[y]);
        const float r = now == -INFINITY ? 0.f : now;
        l *= ex2(high - r);
#pragma unroll
        for (int y = 0; y < 32; ++y) l += ex2(s[y] - r);
        high = now;
        token_powers(t, x0, s);
#pragma unroll
        for (int y = 0; y < 32; ++y) top = fmaxf(top, s[y]);
    }
    top += kRaise;
    const bool need = top > m + kRaise;
    if (first) {
        m = top;
    } else if (__any_sync(0xffffffffu, need)) {
        scale_output(t.to, t.width, need ? ex2(m - top) : 1.f);
        if (need) m = top;
    }
    const float off = kUpBits - (m == -INFINITY ? 0.f : m);
#pragma unroll 1
    for (int x0 = 0; x0 < kN; x0 += 32) {
        float s[32];
        token_scores(t, x0, s);
        token_powers(t, x0, s);
        uint32_t w[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) w[y] = half2_of(ex2(s[2 * y] + off), ex2(s[2 * y + 1] + off));
        tmem_st16(t.ts + x0 / 2, w);
    }
    return make_float3(m, l, high);
}

template <int D, bool QZ, int CV>
__global__ void __launch_bounds__(PCfg<D, QZ, CV>::kThreads, 1) prefix_tc_kernel(const __grid_constant__ Maps maps, const Args a) {
    using C = PCfg<D, QZ, CV>;
    constexpr int kRing = C::kRing, kRaw = C::kRaw;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    enum {
        B_SEG = 0, B_SEGFREE = 2, B_Q = 4, B_S = 6, B_P = 8, B_O = 10, B_ML = 12, B_READ, B_DONE, B_FULL,
        B_EMPTY = B_FULL + kRing, B_RFULL = B_EMPTY + kRing, B_REMPTY = B_RFULL + kRaw, B_N = B_REMPTY + kRaw
    };
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ PSeg segs[2];
    __shared__ uint32_t tmem_base, bad_sm[kBad];
    // QZ: the largest powers of a block's keys and values (biased; in the second byte), and whether its tokens' are in a table
    __shared__ uint32_t power_sm[kBad];
    __shared__ int4 raw_sm[kRaw];            // of a raw block: tokens (< 0: no more blocks), bad boxes, the block's number (>= 0: keys)
    __shared__ int abort_sm;
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    if (tid == 0) {
        auto mbar_init = [](uint32_t at, int count) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(at), "r"(count)); };
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_SEG + i), 1);
            mbar_init(bar(B_SEGFREE + i), 9);            // softmax warps, products
            mbar_init(bar(B_Q + i), 4);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4);
            mbar_init(bar(B_O + i), 1);
        }
        mbar_init(bar(B_ML), 8);
        mbar_init(bar(B_READ), 8);
        mbar_init(bar(B_DONE), 1);
        for (int s = 0; s < kRing; ++s) {
            mbar_init(bar(B_FULL + s), QZ ? 4 : 1);
            mbar_init(bar(B_EMPTY + s), 1);
        }
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(bar(B_RFULL + s), 1);
            mbar_init(bar(B_REMPTY + s), 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_sm = 0;
    }
    wait_for_last_kernel();
    // (QZ: the array's own alignment leaves the last 1024 bytes to the tables)
    if (QZ && sm != smraw) {
        if (tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
        return;
    }
    Start st;
    int share = 1;                           // CTAs of a piece, one for each row item
    if (p.n_seq == 1) {
        int bits = 0;
        const Group gr = group_of<true, kItem>(a, 0, &bits);
        const int64_t tokens = paged_tokens(p, p.kv_len[0]);
        if (bits && tid == 0) atomicOr(&g_status, bits);
        share = gr.RG > 1 && gr.RG <= kPieces / 2 ? gr.RG : 1;
        st.total = tokens == 0 ? 0 : (int64_t)tiles_of<kN>(tokens) * (share > 1 ? p.Hkv : gr.I);
        st.N = (int)min((int64_t)(kPieces / share), st.total);
        st.piece = (int)blockIdx.x / share;
        st.b = 0;
        if (st.piece >= st.N) return;
        st.rem = st.u0 = split_at(st.total, st.N, st.piece);
        st.u1 = split_at(st.total, st.N, st.piece + 1);
    } else if (!find_start<true, C::kThreads, kN, kItem>(a, &st)) {
        return;
    }
    if (warp == C::kMmaWarp) tmem_alloc<512>(smem_u32(&tmem_base));
    // ---- the loader's place: its item and block, and the segment that begins there ----
    int w_b = st.b, w_tokens = 0, w_tiles = 1, w_item = 0, w_t0 = 0, w_page = -1;
    Group w_gr{};
    const int w_box = min(p.page, kN);
    // the page of this lane's box of block t (up to t1)
    auto page_of = [&](int t, int t1) {
        const int pos = t * kN + (lane & 7) * w_box;
        return t < t1 && (lane & 7) * w_box < kN && pos < w_tokens ? paged_page(p, w_b, pos) : -1;
    };
    // the segment from unit u on, as number `seg`, its first stage and block n and blk
    auto make_seg = [&](int64_t u, int seg, int n, int blk) {
        const int t1 = (int)min((int64_t)w_tiles, w_t0 + (st.u1 - u));
        PSeg g;
        g.m0 = w_gr.m0;
        g.r0 = share > 1 ? (int)blockIdx.x % share * kItem : (w_item % w_gr.RG) * kItem;
        g.R = min(kItem, w_gr.rows - g.r0);
        g.hk = share > 1 ? w_item : w_item / w_gr.RG;
        g.nb = t1 - w_t0;
        g.len = w_tokens - w_t0 * kN;
        g.n0 = n;
        g.blk0 = blk;
        g.whole = g.nb == w_tiles;
        g.k = g.np = g.rec = 0;
        if (!g.whole) {
            Seg x;
            place_piece(st, u - w_t0, w_tiles, &x);
            g.k = x.k;
            g.np = x.np;
            g.rec = 2 * (x.c0 * share + (int)blockIdx.x % share) + x.s0;
        }
        segs[seg & 1] = g;
    };
    w_tokens = (int)paged_tokens(p, p.kv_len[w_b]);
    w_gr = group_of<true, kItem>(a, w_b);
    w_tiles = tiles_of<kN>(w_tokens);
    w_item = divide(st.rem, w_tiles, &w_t0);
    // ---- Q rows of tile i, 16 bytes a lane, into the layout that the products read: on their way (those of the first
    // segment while the pages are looked up and TMEM is allocated, before K and V fill the memory's queues) ----
    constexpr int QCH = D / 8, QPER = 32 / QCH;                          // chunks of a row; rows at a time
    const int q_ch = lane % QCH, q_row = (warp & 3) * 32 + lane / QCH;
    auto load_q = [&](int i, int m0, int r0, int R, int hk) {
        const int tile_row = R > kM ? kM * i : 0;
        const uint32_t at = sb + (uint32_t)i * C::kTileBytes + 16384u * (q_ch >> 3);
        const int flat = r0 + tile_row + q_row, seq = flat / p.G;
        int h = flat - seq * p.G;
        const char* src = a.Q.data + ((int64_t)(m0 + seq) * a.Q.row + (int64_t)(hk * p.G + h) * a.Q.head + 8 * q_ch) * 2;
#pragma unroll 1
        for (int x = 0; x < 32; x += QPER) {
            const bool in = tile_row + q_row + x < R;
            cp_async16_z(at + kmaj_chunk(q_row + x, q_ch & 7), in ? src : a.Q.data, in ? 16u : 0u);
            src += (int64_t)QPER * a.Q.head * 2;
            for (h += QPER; h >= p.G; h -= p.G) src += (a.Q.row - (int64_t)p.G * a.Q.head) * 2;
        }
    };
    if (warp == C::kLoadWarp) {
        w_page = page_of(w_t0, w_tiles);
        if (lane == 0) make_seg(st.u0, 0, 0, 0);
    } else if (warp < C::kMmaWarp) {
        const int r0 = share > 1 ? (int)blockIdx.x % share * kItem : (w_item % w_gr.RG) * kItem;
        load_q(warp >> 2, w_gr.m0, r0, min(kItem, w_gr.rows - r0), share > 1 ? w_item : w_item / w_gr.RG);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tb = tmem_base;

    auto wait = [&](int i, uint32_t parity) -> bool { return ring_wait(bar(i), parity & 1u, &abort_sm); };
    auto wait_all = [&](int i, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(i, parity)); };
    auto get_seg = [&](int n, PSeg* g) -> bool {
        if (!wait(B_SEG + (n & 1), (uint32_t)(n >> 1))) return false;
        *g = segs[n & 1];
        return g->nb >= 0;
    };
    // Blocks are loaded, and read by the products, in one order: `look` blocks of K, then by turns V of a block and K of
    // the one `look` further on.  Stage n is the n-th of them over all segments.
    auto stage_at = [&](int n) { return (uint32_t)(2 + n % kRing) * C::kTileBytes; };
    auto look_of = [](const PSeg& g) { return g.R > kM ? 1 : 2; };

    if (warp >= C::kMmaWarp) {
        if constexpr (C::kOtherRegs < 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp == C::kLoadWarp) {
            // ================================ pages and loads ================================
            const int box = w_box, lb = 31 - __clz(box), nbox = kN >> lb;               // tokens of a box, boxes of a block
            const int half = lane >> 3, by = (lane & 7) << lb;                         // this lane's box (half: 64 channels)
            int64_t u = st.u0;
            int seg = 0, n = 0, blk = 0;
            bool ok = true;
            uint32_t wrong = 0;
            while (u < st.u1 && ok) {
                if (seg >= 2 && !(ok = wait_all(B_SEGFREE + (seg & 1), (uint32_t)(seg / 2 - 1)))) break;
                if (seg > 0 && lane == 0) make_seg(u, seg, n, blk);
                const int t0 = w_t0, t1 = (int)min((int64_t)w_tiles, t0 + (st.u1 - u)), nb = t1 - t0, tokens = w_tokens;
                const int r0 = share > 1 ? (int)blockIdx.x % share * kItem : (w_item % w_gr.RG) * kItem;
                const int hk = share > 1 ? w_item : w_item / w_gr.RG, look = w_gr.rows - r0 > kM ? 1 : 2;
                if (lane == 0) mbar_arrive1(bar(B_SEG + (seg & 1)));
                if (p.kv_len[w_b] > tokens) wrong = 1;
                // the page of this lane's box of the next block, and of those that wait for their V
                int next = seg == 0 ? (t0 < t1 ? w_page : -1) : page_of(t0, t1), now = -1, held[2] = {-1, -1};
                ++seg;
                const bool give_up = gives_up(a.give_up, blk, nb);
                const int stop = give_up ? a.give_up - blk : nb + look;
                for (int x = 0; x < stop && ok; ++x) {
                    held[1] = held[0];
                    held[0] = now;
                    now = next;
                    next = page_of(t0 + x + 1, t1);
#pragma unroll
                    for (int kv = 1; kv >= 0; --kv) {
                        const int t = t0 + (kv ? x - look : x);
                        if (kv ? x < look : x >= nb) continue;
                        const int page = kv ? (look == 1 ? held[0] : held[1]) : now, pos = t * kN + by, at = pos & (p.page - 1);
                        const bool used = (lane & 7) < nbox && pos < tokens, bad = used && page < 0;
                        const uint32_t bad_mask = __ballot_sync(0xffffffffu, bad) & 0xffu;
                        if (bad_mask) wrong = 1;
                        if constexpr (QZ) {
                            const int r = n % kRaw, good = __popc(__ballot_sync(0xffffffffu, used) & 0xffu) - __popc(bad_mask);
                            if (n >= kRaw && !(ok = wait_all(B_REMPTY + r, (uint32_t)(n / kRaw - 1)))) break;
                            if (lane == 0) {
                                if (!kv) bad_sm[blk % kBad] = bad_mask;
                                raw_sm[r] = make_int4(min(kN, tokens - t * kN), (int)bad_mask, (kv ? t - t0 : blk), kv);
                                mbar_expect(bar(B_RFULL + r), (uint32_t)(good * box * (D + 1 + !kv)));
                            }
                            __syncwarp();
                            if (used && !bad && half < 3 - kv) {
                                const int64_t row = ((int64_t)page * p.Hkv + hk) * p.page + at;
                                const uint32_t dst = sb + (2 + kRing) * C::kTileBytes + r * C::kRawBytes;
                                if (half == 0) bulk_load(dst + by * D, (kv ? p.V : p.K) + row * D, (uint32_t)(box * D), bar(B_RFULL + r));
                                else bulk_load(dst + kN * (D + half - 1) + by, (kv || half == 2 ? p.Vs : p.Ks) + row, (uint32_t)box, bar(B_RFULL + r));
                            }
                        } else {
                            // (a box behind the prefix' tokens or on a bad page is read behind the pool's end, as zeros)
                            const int s = n % kRing;
                            if (n >= kRing && !(ok = wait_all(B_EMPTY + s, (uint32_t)(n / kRing - 1)))) break;
                            if (lane == 0) {
                                if (!kv) bad_sm[blk % kBad] = bad_mask;
                                mbar_expect(bar(B_FULL + s), C::kTileBytes);
                            }
                            __syncwarp();
                            if ((lane & 7) < nbox && half < D / 64)
                                tma_load4(sb + stage_at(n) + 16384u * half + 128u * by, kv ? &maps.v : &maps.k, 0, at, half,
                                          page < 0 ? p.n_pages * p.Hkv : page * p.Hkv + hk, bar(B_FULL + s));
                        }
                        ++n;
                        blk += !kv;
                    }
                }
                if (give_up) {
                    if (lane == 0) *reinterpret_cast<volatile int*>(&abort_sm) = 1;
                    ok = false;
                }
                u += nb;
                w_t0 = 0;
                if (++w_item == (share > 1 ? p.Hkv : w_gr.I) && u < st.u1) {
                    w_item = 0;
                    do {                                               // (units are left: there is such a prefix)
                        ++w_b;
                        w_tokens = (int)paged_tokens(p, p.kv_len[w_b]);
                        w_gr = group_of<true, kItem>(a, w_b);
                    } while (w_tokens == 0 || w_gr.I == 0);
                    w_tiles = tiles_of<kN>(w_tokens);
                }
            }
            // the others' end
            if (ok && seg >= 2) ok = wait_all(B_SEGFREE + (seg & 1), (uint32_t)(seg / 2 - 1));
            for (int x = n; x < n + CV && ok; ++x)
                if (x >= kRaw) ok = wait_all(B_REMPTY + x % kRaw, (uint32_t)(x / kRaw - 1));
            if (lane == 0) {
                if (ok) {
                    segs[seg & 1].nb = -1;
                    mbar_arrive1(bar(B_SEG + (seg & 1)));
                }
                // leave no copy in flight (before the end of the codes, which is one more phase of its barrier)
                constexpr int kLast = QZ ? kRaw : kRing, kFirst = QZ ? (int)B_RFULL : (int)B_FULL;
                for (int x = max(0, n - kLast); x < n; ++x) mbar_wait(bar(kFirst + x % kLast), (uint32_t)(x / kLast) & 1u, kWaitNs);
                for (int x = n; x < n + CV && ok; ++x) {
                    raw_sm[x % kRaw] = make_int4(-1, 0, 0, 0);
                    mbar_arrive1(bar(B_RFULL + x % kRaw));
                }
                if (wrong) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
            }
            __syncwarp();
        } else if (warp == C::kMmaWarp) {
            // ================================ products ================================
            if (lane == 0) {
                // (QZ: float16 operands)
                constexpr uint32_t kind = QZ ? ~((1u << 7) | (1u << 10)) : ~0u;
                constexpr uint32_t id_s = idesc_bf16(kM, kN, 0) & kind, id_o = idesc_bf16(kM, D, 1) & kind;
                constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
                PSeg g;
                bool ok = true;
                int n = 0, np[2] = {0, 0}, nq[2] = {0, 0};             // stages; weights and Q tiles that were waited for
                auto full = [&](int x) { return wait(B_FULL + x % kRing, (uint32_t)(x / kRing)); };
                auto s_mma = [&](int i, int x) {
                    const uint32_t q = desc_lo(sb + (uint32_t)i * C::kTileBytes, 16), k = desc_lo(sb + stage_at(x), 16);
#pragma unroll
                    for (int y = 0; y < D / 16; ++y) {
                        const uint32_t o = (uint32_t)(y >> 2) * 1024u + (uint32_t)(y & 3) * 2u;   // 16-byte units
                        mma_ss(tb + C::TS(i), q + o, k + o, hi, id_s, y > 0);
                    }
                    mma_commit(bar(B_S + i));
                };
                for (int seg = 0; ok && get_seg(seg, &g); ++seg) {
                    mbar_arrive1(bar(B_SEGFREE + (seg & 1)));
                    const bool two = g.R > kM;
                    const int look = look_of(g);
                    for (int x = 0; x < min(look, g.nb) && ok; ++x, ++n) {
                        ok = full(n);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (ok && (two || i == x)) {
                                ok = wait(B_Q + i, (uint32_t)nq[i]++);
                                fence_after();
                                if (ok) s_mma(i, n);
                            }
                        mma_commit(bar(B_EMPTY + n % kRing));
                    }
                    for (int j = 0; j < g.nb && ok; ++j) {
                        const bool more = j + look < g.nb;
                        ok = full(n);
                        const uint32_t v = desc_lo(sb + stage_at(n), 16384);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (ok && (two || i == (j & 1))) {
                                if (!(ok = wait(B_P + i, (uint32_t)np[i]++))) break;
                                fence_after();
#pragma unroll
                                for (int y = 0; y < kN / 16; ++y)
                                    mma_ts(tb + C::TO(i), tb + C::TS(i) + 8 * y, v + 128u * y, hi, id_o, y > 0 ? 1u : (uint32_t)(j >= look));
                                const bool last = !two || i == 1;                  // (tile of the block)
                                if (last) mma_commit(bar(B_EMPTY + n % kRing));
                                if (!more) {
                                    mma_commit(bar(B_O + i));
                                } else {
                                    if (!(ok = full(n + 1))) break;
                                    s_mma(i, n + 1);
                                    if (last) mma_commit(bar(B_EMPTY + (n + 1) % kRing));
                                }
                            }
                        n += 1 + more;
                    }
                }
                // leave no product in flight
                mma_commit(bar(B_DONE));
                if (!mbar_wait(bar(B_DONE), 0, kWaitNs)) abort_sm = 1;
            }
            __syncwarp();
        } else if (QZ && warp >= C::kConvWarp) {
            // ================================ codes to float16 ================================
            const int t = tid & 127;
            // CV == 1: of the blocks (two at most) whose keys are converted and whose values are not, the oldest first: largest
            // power of the values, whether they lie apart, 512
            uint32_t values = 0u;
            for (int n = CV == 1 ? 0 : (warp - C::kConvWarp) >> 2;; n += CV) {
                const int r = n % kRaw, s = n % kRing;
                if (!wait_all(B_RFULL + r, (uint32_t)(n / kRaw))) break;
                const int4 info = raw_sm[r];
                if (info.x < 0) break;
                if (n >= kRing && !wait_all(B_EMPTY + s, (uint32_t)(n / kRing - 1))) break;
                const uint8_t* raw = sm + (size_t)(2 + kRing) * C::kTileBytes + (size_t)r * C::kRawBytes;
                uint8_t* out = sm + stage_at(n);
                const int lb = 31 - __clz(min(p.page, kN));
                const bool some = info.x < kN || info.y;
                auto hidden = [&](int k) { return k >= info.x || (info.y >> (k >> lb)) & 1; };
                // the largest of 128 powers, of tokens that are seen, and whether others are further below it than `most`
                struct Range {
                    uint32_t top;
                    bool wide;
                };
                auto range = [&](const uint8_t* powers, int most) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(powers + 4 * lane);
                    auto largest = [](uint32_t x) { return max(max(x & 255u, (x >> 8) & 255u), max((x >> 16) & 255u, x >> 24)); };
                    auto smallest = [](uint32_t x) { return min(min(x & 255u, (x >> 8) & 255u), min((x >> 16) & 255u, x >> 24)); };
                    uint32_t hi = largest(w), lo = smallest(w);
                    if (some) {
                        const int left = info.x - 4 * lane;
                        const uint32_t seen = hidden(4 * lane) ? 0u : left < 4 ? (1u << (8 * left)) - 1u : ~0u;
                        hi = largest(w & seen);
                        lo = smallest(w | ~seen);
                    }
                    hi = __reduce_max_sync(0xffffffffu, hi);
                    return Range{hi, (bool)__any_sync(0xffffffffu, (int)(hi - lo) > most)};
                };
                Range E;
                if (info.w && CV == 1) {
                    // (these four warps have converted the block's keys, in the same order as the values)
                    E = Range{values & 255u, (bool)(values & 256u)};
                    values >>= 16;
                } else {
                    E = range(raw + kN * D, info.w ? kApartValues : kApartKeys);
                }
                if (!info.w) {
                    const Range F = range(raw + kN * (D + 1), kApartValues);
                    const bool table = E.wide || F.wide;
                    if (t == 0) power_sm[info.z % kBad] = E.top | F.top << 8 | (uint32_t)table << 16;
                    if (table && t < kWarp) {
                        // (powers that the block's numbers do not have in them)
                        uint32_t* to = reinterpret_cast<uint32_t*>(sm + C::kTableAt + info.z % kTables * kTableBytes) + lane;
                        to[0] = E.wide ? *reinterpret_cast<const uint32_t*>(raw + kN * D + 4 * lane) : E.top * 0x01010101u;
                        to[kN / 4] = F.wide ? *reinterpret_cast<const uint32_t*>(raw + kN * (D + 1) + 4 * lane) : F.top * 0x01010101u;
                    }
                    const uint32_t next = F.top | (uint32_t)F.wide << 8 | 512u;
                    values = values & 512u ? values & 0xffffu | next << 16 : next;
                }
                // 16 codes a thread: CH such chunks a token, a warp takes PT tokens of every 128 / CH.  Each lane finds one
                // token's factor, 2^(e - E) in float16: down to 2^-14, then 2^-15.  (Loads before stores, which might be the same
                // place for all the compiler knows: a block took one warp a scheduler 1190 clocks, now 560.)
                constexpr int CH = D / 16, PT = 32 / CH, kBatch = 4;
                const int own = 128 / CH * (lane / PT) + PT * (warp & 3) + lane % PT;
                // (of tokens that are not seen: anything)
                const int down = E.wide ? 0 : min(max(0, (int)E.top - (int)raw[kN * D + own]), 15);
                const uint32_t factor = (down < 15 ? (15u - down) << 10 : 1u << 9) * 0x10001u;
#pragma unroll
                for (int x0 = 0; x0 < CH; x0 += kBatch) {
                    uint4 w[kBatch];
#pragma unroll
                    for (int x = 0; x < kBatch; ++x) {
                        w[x] = *reinterpret_cast<const uint4*>(raw + (size_t)(t + 128 * (x0 + x)) * 16);
                        if (some && hidden((t + 128 * (x0 + x)) / CH)) w[x] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int x = 0; x < kBatch; ++x) {
                        const int e = t + 128 * (x0 + x), k = e / CH, c = e % CH;
                        const uint32_t f = __shfl_sync(0xffffffffu, factor, PT * (x0 + x) + lane / CH);
                        const uint32_t in[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
                        uint32_t z[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            widen(in[i], z[2 * i], z[2 * i + 1]);
                            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(z[2 * i]) : "r"(f));
                            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(z[2 * i + 1]) : "r"(f));
                        }
                        const uint4 y0 = make_uint4(z[0], z[1], z[2], z[3]), y1 = make_uint4(z[4], z[5], z[6], z[7]);
                        uint8_t* row = out + 16384 * (c >> 2) + k * 128;
                        const int c16 = 2 * (c & 3);
                        const bool swap = D == 128 && (c & 4);         // (so that eight lanes' 16 bytes lie in different banks)
                        *reinterpret_cast<uint4*>(row + (((c16 + swap) ^ k) & 7) * 16) = swap ? y1 : y0;
                        *reinterpret_cast<uint4*>(row + (((c16 + !swap) ^ k) & 7) * 16) = swap ? y0 : y1;
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive1(bar(B_FULL + s));
                    mbar_arrive1(bar(B_REMPTY + r));
                }
            }
        }
    } else {
        // ================================ softmax ================================
        if constexpr (C::kSoftmaxRegs > C::kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;                    // tile, row of the tile
        const uint32_t lo = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tb + lo + C::TS(i), to = tb + lo + C::TO(i);
        float c = a.scale_log2;                                                 // (QZ: with the power of two of the row of Q)
        uint8_t* Qt = sm + (size_t)i * C::kTileBytes;
        int ns = 0, no = 0, pairs = 0;                                          // blocks, segments with blocks, and with two halves
        for (int it = 0;; ++it) {
            PSeg g;
            if (!__all_sync(0xffffffffu, get_seg(it, &g))) break;
            if (lane == 0) mbar_arrive1(bar(B_SEGFREE + (it & 1)));
            const bool two = g.R > kM, pair = !two && g.nb > 1;
            const int n = two ? g.nb : (g.nb + 1 - i) / 2, look = look_of(g);
            const int tile_row = two ? kM * i : 0;
            if (n > 0) {
                // ---- Q rows of the tile ----
                if (it > 0) {
                    // (a tile without blocks in the first segment has not waited for its rows' copies there, and copies of one
                    // thread land in any order)
                    cp_async_wait_all();
                    load_q(i, g.m0, g.r0, g.R, g.hk);
                }
                cp_async_wait_all();
                if constexpr (QZ) {
                    // float16 numbers, the row's largest magnitude in [2^14, 2^15)
#pragma unroll 4
                    for (int x = 0; x < 32; x += QPER) {
                        uint4* at = reinterpret_cast<uint4*>(Qt + 16384 * (q_ch >> 3) + kmaj_chunk(q_row + x, q_ch & 7));
                        const uint4 z = *at;
                        uint32_t w[4] = {z.x, z.y, z.z, z.w}, big = 0u;
#pragma unroll
                        for (int y = 0; y < 4; ++y) big = max(big, max((w[y] << 16) & 0x7fff0000u, w[y] & 0x7fff0000u));
#pragma unroll
                        for (int o = 1; o < QCH; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                        const uint32_t up = min(268u - (big >> 23), 240u);
                        const float f = __uint_as_float(up << 23);
#pragma unroll
                        for (int y = 0; y < 4; ++y) w[y] = half2_of(__uint_as_float(w[y] << 16) * f, __uint_as_float(w[y] & 0xffff0000u) * f);
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                        // (rows x .. x + QPER - 1 of the warp's 32 are those of lanes x ..)
                        const uint32_t mine = __shfl_sync(0xffffffffu, up, ((lane - x) * QCH) & 31);
                        if (lane >= x && lane < x + QPER) c = a.scale_log2 * __uint_as_float((254u - mine) << 23);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bar(B_Q + i));
            }
            float m = -INFINITY, l = 0.f;
            [[maybe_unused]] float ml = -INFINITY;                              // QZ: the largest score, against which l is kept
            bool ok = true;
            for (int jj = 0; jj < n && ok; ++jj) {
                const int j = two ? jj : 2 * jj + i;
                if (!(ok = wait_all(B_S + i, (uint32_t)(ns + jj)))) break;
                fence_after();
                constexpr int kHeld = C::kHeld;
                float s[kHeld];
                const int valid = g.len - j * kN;
                const uint32_t bad = bad_sm[(g.blk0 + j) % kBad];
                const bool some = valid < kN || bad;
                const int lb = 31 - __clz(min(p.page, kN));
                // columns x0 .. x0 + 31 in s[at ..] (rare: a branch, and not conditions in every block's path)
                auto hide = [&](int at, int x0) {
                    if (!some) return;
                    asm volatile("" ::: "memory");
                    const uint32_t seen = seen_columns(x0, valid, bad, lb);
#pragma unroll
                    for (int x = 0; x < 32; ++x) s[at + x] = (seen >> x) & 1u ? s[at + x] : -INFINITY;
                };
                auto weighed = [&] {
                    tmem_wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(bar(B_P + i));
                };
                [[maybe_unused]] uint32_t powers = 0u;
                if constexpr (QZ) {
                    powers = power_sm[(g.blk0 + j) % kBad];
                    if (powers >> 16) {
                        const uint32_t table = sb + C::kTableAt + (uint32_t)((g.blk0 + j) % kTables) * kTableBytes;
                        const float3 x = by_token_block(ByToken{ts, to, table, bad, c, valid, lb, D}, jj == 0, make_float3(m, l, ml));
                        m = x.x, l = x.y, ml = x.z;
                        weighed();
                        continue;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int x0 = kN - kHeld; x0 >= 0; x0 -= kHeld) {
#pragma unroll
                    for (int x = 0; x < kHeld; x += 32) tmem_ld32(ts + x0 + x, s + x);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < kHeld; x += 32) hide(x, x0 + x);
#pragma unroll
                    for (int x = 0; x < kHeld; ++x) mx[x & 3] = fmaxf(mx[x & 3], s[x]);
                }
                if (!QZ && valid < kN) {
                    // values behind the prefix, which may be anything, become zero (both tiles see to it)
                    const int vs = g.n0 + j + min(g.nb, j + look);
                    if (!(ok = wait_all(B_FULL + vs % kRing, (uint32_t)(vs / kRing)))) break;
                    for (int x = max(valid, 0) * 8 + r; x < kN * 8; x += kM)
#pragma unroll
                        for (int y = 0; y < D / 64; ++y) *reinterpret_cast<uint4*>(sm + stage_at(vs) + 16384 * y + 16 * x) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                }
                // the scores' factor, and what their weights' exponents have besides
                float cb = c, add = 0.f;
                const float largest = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if constexpr (QZ) {
                    // (0 would make NaN of hidden scores, an infinity of those that are 0)
                    cb = fminf(fmaxf(c * __uint_as_float((powers & 255u) << 23), 1.2e-38f), 3.0e38f);
                    add = (float)(int)(powers >> 8) - 127.f;
                }
                const float top = fmaf(largest, cb, add + kRaise);
                const bool need = top > m + kRaise;
                if (jj == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, need)) {
                    // (O is quiet: S of this block was issued behind the tile's last P V, and is done)
                    const float f = need ? ex2(m - top) : 1.f;
                    if (!QZ) l *= f;
                    scale_output(to, D, f);
                    if (need) m = top;
                }
                const float base = m == -INFINITY ? 0.f : m;
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                float off = QZ ? add + kUpBits - base : -base;
                // (QZ: a block whose weights are nothing beside m still counts in l: numbers that float16 takes to 0)
                const float high = largest * cb;
                if (QZ && high + add < base - 60.f && high > -INFINITY) off = -high - 40.f;
                const float2 c2 = make_float2(cb, cb), b2 = make_float2(off, off);
                // weights of the 32 scores in s[at ..], columns x on, over the scores
                auto weigh = [&](int at, int x) {
                    uint32_t pw[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        float2 e = fma2(make_float2(s[at + 2 * y], s[at + 2 * y + 1]), c2, b2);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        ls[y & 1] = add2(ls[y & 1], e);
                        pw[y] = QZ ? half2_of(e.x, e.y) : pack2(e.x, e.y);
                    }
                    tmem_st16(ts + x / 2, pw);
                };
                if constexpr (kHeld < kN) {
#pragma unroll 1
                    for (int x = 0; x < kN; x += 32) {
                        weigh(0, x);
                        if (x + 32 < kN) {
                            tmem_ld32(ts + x + 32, s);
                            tmem_wait_ld();
                            hide(0, x + 32);
                        }
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < kN; x += 32) weigh(x, x);
                }
                const float sum = (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                if constexpr (QZ) {
                    const float now = fmaxf(ml, high), r = now == -INFINITY ? 0.f : now;
                    l *= ex2(ml - r);
                    if (sum != 0.f) l = fmaf(sum, ex2(-off - r), l);
                    ml = now;
                } else {
                    l += sum;
                }
                weighed();
            }
            // ---- the segment's part: for the row, m, l and O ----
            if (n > 0 && ok) ok = wait_all(B_O + i, (uint32_t)no);
            if (!ok) break;
            fence_after();
            ns += n;
            no += n > 0;
            // QZ: O is in the weights' unit, 2^{m - 15}, l in the scores', 2^ml: the factor from one to the other, which may be
            // far from one, by its square root
            [[maybe_unused]] auto root = [](float m, float ml) {
                return m == -INFINITY ? 0.f : ex2(0.5f * (m - kUpBits - (ml == -INFINITY ? 0.f : ml)));
            };
            float f0 = QZ ? root(m, ml + kRoom) : 1.f, f1 = 0.f;
            if constexpr (QZ) {
                if (pair) {
                    // both halves' m and l, in the place of their Q rows
                    reinterpret_cast<float4*>(Qt)[r] = make_float4(m, l, ml, 0.f);
                }
            } else if (pair) {
                reinterpret_cast<float2*>(Qt)[r] = make_float2(m, l);
            }
            if (pair) {
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bar(B_ML));
                if (!wait_all(B_ML, (uint32_t)pairs)) break;
                fence_after();                                                  // (the other half's O is read here too)
                if constexpr (QZ) {
                    const float4 x = reinterpret_cast<const float4*>(sm)[r], y = reinterpret_cast<const float4*>(sm + C::kTileBytes)[r];
                    ml = fmaxf(x.z, y.z);
                    const float base = ml == -INFINITY ? 0.f : ml;
                    l = ex2(x.z - base) * x.y + ex2(y.z - base) * y.y;
                    f0 = root(x.x, ml + kRoom);
                    f1 = root(y.x, ml + kRoom);
                } else {
                    const float2 x = reinterpret_cast<const float2*>(sm)[r], y = reinterpret_cast<const float2*>(sm + C::kTileBytes)[r];
                    m = fmaxf(x.x, y.x);
                    const float base = m == -INFINITY ? 0.f : m;
                    f0 = ex2(x.x - base);
                    f1 = ex2(y.x - base);
                    l = f0 * x.y + f1 * y.y;
                }
            }
            if (QZ) {
                m = ml + kRoom;
                l *= ex2(-kRoom);
            }
            const int row = tile_row + r, flat = g.r0 + row, seq = flat / p.G;
            const bool mine = row < g.R && n > 0;
            const Parts& q = a.parts;
            const int64_t at = (int64_t)(g.m0 + seq) * p.Hq + g.hk * p.G + flat - seq * p.G;
            float* rec = q.rec + ((int64_t)blockIdx.x * 2 + (g.k == 0 ? g.rec & 1 : 0)) * part_record(kItem, D);
            // (two halves: half of the columns each)
            const int c0 = pair ? i * (D / 2) : 0, c1 = pair ? c0 + D / 2 : D;
            if (n > 0) {
#pragma unroll 1
                for (int x = c0; x < c1; x += 32) {
                    float o[32];
                    if (pair) {
                        float z[32];
                        tmem_ld32(tb + lo + C::TO(0) + x, o);
                        tmem_ld32(tb + lo + C::TO(1) + x, z);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] = QZ ? fmaf(f0 * o[y], f0, f1 * z[y] * f1) : fmaf(f0, o[y], f1 * z[y]);
                    } else {
                        tmem_ld32(to + x, o);
                        tmem_wait_ld();
                        if (QZ) {
#pragma unroll
                            for (int y = 0; y < 32; ++y) o[y] = o[y] * f0 * f0;
                        }
                    }
                    if (mine) {
#pragma unroll
                        for (int y = 0; y < 32; y += 4) {
                            float* dst = g.whole ? q.whole + at * D + x + y : rec + ((x + y) / 4 * kItem + row) * 4;
                            *reinterpret_cast<float4*>(dst) = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
                        }
                    }
                }
            }
            if (mine && c0 == 0) {
                if (g.whole) {
                    q.ml[at] = make_float2(m, l);
                } else {
                    rec[kItem * D + row] = m;
                    rec[kItem * D + kItem + row] = l;
                }
                if (g.whole || g.k == 0) q.desc[at] = g.whole ? make_int4(1, 0, 0, 0) : make_int4(g.np, g.rec, row, share);
            }
            fence_before();
            if (pair) {
                __syncwarp();
                if (lane == 0) mbar_arrive1(bar(B_READ));
                if (!wait_all(B_READ, (uint32_t)pairs)) break;
                ++pairs;
            }
        }
        cp_async_wait_all();                 // (the first Q rows, where a wait gave up before them)
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (abort_sm && tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
    if (warp == C::kMmaWarp) tmem_dealloc<512>(tb);
}

template <int D, bool QZ, int CV> cudaError_t launch_tc(const DecodeArgs& d, cudaStream_t st) {
    using C = PCfg<D, QZ, CV>;
    static std::atomic<uint64_t> done{0};
    Maps maps{};
    if constexpr (!QZ) {
        const int64_t depth = (int64_t)d.p.n_pages * d.p.Hkv;
        const int rows = d.p.page < kN ? d.p.page : kN;
        if (!make_tmap_pages(&maps.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d.p.K, D, d.p.page, depth, rows, 1) ||
            !make_tmap_pages(&maps.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d.p.V, D, d.p.page, depth, rows, 1))
            return cudaErrorInvalidValue;
    }
    cudaError_t e = opt_in_smem(prefix_tc_kernel<D, QZ, CV>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_behind(prefix_tc_kernel<D, QZ, CV>, kPieces, C::kThreads, C::kSmem, st, maps, make_args(d));
}

}  // namespace

cudaError_t launch_prefix_tc(const DecodeArgs& a, cudaStream_t st) {
    if (!a.p.Ks) return a.p.d == 128 ? launch_tc<128, false, 0>(a, st) : launch_tc<64, false, 0>(a, st);
    if (a.p.d == 64) return launch_tc<64, true, 1>(a, st);
    // One tile of rows whatever the prefixes' sequences are: half of the softmax, and the conversion is what counts (32
    // sequences with up to 100 tokens of their own behind 131072, 32/8 heads, the whole call: 120 us, 127 with four
    // converting warps).
    return (int64_t)a.sh.n_seq * a.p.G <= kM ? launch_tc<128, true, 2>(a, st) : launch_tc<128, true, 1>(a, st);
}

cudaError_t prefix_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
