// K8 (bf16, tensor cores): causal softmax attention over packed prompts, keys and values packed too or in
// the pages of a cache.
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j <= i + Lk - Lq.  One pass over
// the keys in blocks of 128 with a running maximum m and sum l per row (log2 units):
//   S = Q K^T,  P = 2^{c S - m},  l += sum P,  O += P V,      o = O / l,
// m is raised lazily: it is set 8 above a maximum (log2 units), and O and l are rescaled (in TMEM) only when a
// later block's maximum passes it, so that blocks rarely wait for O.  No weight is above one, as with the maximum
// itself, so that O does not pass float32 where the values do not.
//
// An item is 256 queries of one head, two tiles of 128 (MMA M = 128, TMEM lane = query) that share every
// K and V block; while the tensor core works for one tile, the other tile's softmax runs.  Short
// sequences take one tile an item and two CTAs per SM instead, each in half an SM (see one_tile below).
// A CTA goes from item to item, taking over blocks of the grid that have not started (cluster launch
// control), so that an item's lookup, first loads and last stores run beside its neighbours' products;
// barrier phases, ring places and tile counts run on over the items.  Warps (of two tiles):
//   * 11 (items): the next block, its sequence and tile, published one item ahead;
//   * 9 (loader): Q, K and V tiles by TMA, 128-byte swizzle, into a ring of K and V blocks;
//   * 8 (MMA, one thread): per block and tile O_i += P_i V_j, then S_i = Q_i K_{j+1}^T.  P_i
//     (bf16, read from TMEM as the A operand) lies over S_i's columns: the products of one thread
//     run in order, so S_i of the next block cannot overtake the read of P_i;
//   * 0-3, 4-7 (softmax of tile 0, 1; one thread per query): the row of S into registers,
//     mask on the blocks that some row does not see whole, maximum, weights, P into TMEM, and at the
//     end the rows of o;
//   * 10 (cleaner): on those same blocks, V rows behind the sequence and values that are not finite
//     are zeroed in shared memory before the product (0 x NaN would reach rows that do not see
//     them); the values taken out are added back in the epilogue, for the rows that see them.
// What bounds it: for long sequences the tensor core and its power (16 heads of 32768 tokens, d = 128:
// 2.53 ms, 1740 TFLOP/s, 94 % of the measured bf16 product, and 2.66 ms in a row at 1.8 GHz and the power
// limit; 4 x 4096 x 32 heads 389 us, 1413 TFLOP/s, and 403-420 us in a row): a block pair's products take about 2300 cycles of the issuing thread's 2700, the rest is its wait for
// the weights (a softmax is 1100 cycles, behind it the other tile's products).  At d = 64 the
// exponentials weigh twice as much against the products, whose narrow half (N = 64) runs at half rate (1050
// TFLOP/s); no unit is then above 60 % of its rate, the softmax warps' own dependences are the bound.  Short
// sequences are bound by an item's own chain: scores, weights, product, epilogue.
// Tried and slower: releasing P in halves, comparing S by column groups while it loads, one MMA thread
// for each tile (their products interleave, 9 %), the next pair's waits between the products, one block
// per CTA without taking over others (4 x 4096 x 32 heads 457 against 412 us, ragged prompts 362 against
// 332), all sequences' longest tiles first (their K and V no longer fit L2 together: 427), and at d = 64 three
// places for the scores of both tiles, the next ones issued before the weights are there (one prompt of 32768,
// 16 heads: 2.30 ms against 2.12).
// Keys in pages: the loader's lanes look a block's pages up while its place in the ring is still being read and
// load a box each.  Pages of 64 tokens and more cost next to nothing (512 queries behind 6000 keys, 4 times, 32/8
// heads, d = 128: 198 us, packed rows 192); pages of 16 are 32 boxes of 2 KB a block (280 us).
// The tensor core cuts its float32 sums off instead of rounding them: outputs are low by up to 1e-5 of their
// magnitude at 4096 keys, 1e-4 at 32768 and 5.5e-4 at 131072, where bfloat16 rounds by up to 2^-8.
// Every wait is bounded (1 s, those that may last a whole item 10 s, then LOLA_ATTN_TIMEOUT).
#include <cuda.h>

#include <cmath>

#include "lola_attn.cuh"
#include "lola_attn_mma.cuh"

namespace lola {
namespace {

using namespace tc;

__device__ int32_t g_status;

constexpr int kM = 128;                  // queries per tile
constexpr int kN = 128;                  // keys per block
constexpr int kClean = 4;                // barriers of the blocks to be cleaned
constexpr float kRaise = 8.0f;           // m is set this far above a block's maximum (log2), and raised when one passes it
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kItemNs = 10000000000ull;   // ... of the waits that may last a whole item

// NT: query tiles of a CTA.  Two: one CTA per SM, K and V blocks shared by 256 queries.  One: two CTAs
// per SM, each with its own ring (half the shared memory, half of TMEM).
template <int D, int NT> struct Cfg {
    static constexpr int kQ = NT * kM;                     // queries per item
    static constexpr int kThreads = (NT + 1) * 128;
    static constexpr int kMmaWarp = 4 * NT, kLoadWarp = kMmaWarp + 1, kItemWarp = kMmaWarp + 3;   // (kMmaWarp + 2: the cleaner)
    static constexpr int kTileBytes = kM * D * 2;          // a Q tile, a K block or a V block
    static constexpr int kCap = NT == 2 ? (D == 128 ? 2 : 4) : (D == 128 ? 1 : 2);      // pairs in the ring
    static constexpr int kStageBytes = kM * 64;            // 32 columns of a tile's output
    static constexpr int kSmem = (NT + 2 * kCap) * kTileBytes + NT * kStageBytes + 1024;
    static constexpr int kTmem = 256 * NT;                 // columns
    __device__ static constexpr uint32_t TS(int i) { return 128u * i; }            // S (P over its first half)
    __device__ static constexpr uint32_t TO(int i) { return 128u * NT + (uint32_t)D * i; }
};

struct Maps {
    CUtensorMap q, k, v;   // [rows][heads][d], boxes of 128 rows x 1 head x 64 channels; or k, v of the pools:
                           // [pages x heads][64 channels][page], boxes of up to 128 rows of one page
};


__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two bfloat16 numbers of the larger magnitudes (signs of no meaning); NaN if either is one
__device__ __forceinline__ uint32_t max_abs2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// One item: a query tile (or two) of one head.
struct Item {
    int b, q0, lq, k0, lk, r0, h, live;
};
// The blocks of 128 keys that its tiles read (nb, the most of them nmax) and those that all its rows see
// whole (nf).
template <int NT> struct Span {
    int nb[NT], nmax, nf;
    __device__ __forceinline__ explicit Span(const Item& t) {
        nmax = 0;
        nf = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int first = t.r0 + kM * i, last = min(first + kM, t.lq) - 1, shift = t.lk - t.lq;   // the tile's rows
            nb[i] = first < t.lq ? (max(0, min(t.lk, last + shift + 1)) + kN - 1) / kN : 0;
            if (nb[i] > 0) nf = min(nf, max(0, min(t.lk, first + shift + 1)) / kN);
            nmax = max(nmax, nb[i]);
        }
    }
};

// Query tiles of ROWS rows, found by one warp: the sequences' tiles are counted in order and taken
// backwards (a sequence's longest tiles first, the first sequence's shortest ones at the very end), 32
// sequences in the lanes at a time.  A CTA that takes blocks over finds them in order as a rule, but nothing
// promises it: the lanes go on to other sequences in either direction.
template <int ROWS, bool PG> struct Finder {
    int q0, lq, k0, lk;      // this lane's sequence of the 32 from cb on
    int cb, own, inc;        // ... its tiles, and the tiles up to it in the lanes
    int before, total;       // tiles before cb, tiles of all
    int bits;                // what is wrong with offsets and lengths

    __device__ __forceinline__ int look(const AttnArgs& a, int b) {
        q0 = lq = k0 = lk = 0;
        if (b < 0 || b >= a.n_seq) return 0;
        seq_rows(a.cu_q, b, a.total_q, &q0, &lq, &bits);
        seq_keys<PG>(a, b, &k0, &lk, &bits);
        return (lq + ROWS - 1) / ROWS;
    }
    __device__ __forceinline__ void chunk(const AttnArgs& a, int lane) {
        own = inc = look(a, cb + lane);
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
    }
    __device__ __forceinline__ void start(const AttnArgs& a, int lane) {
        bits = 0;
        cb = (a.n_seq - 1) / kWarp * kWarp;
        int64_t sum = 0;
        for (int b = 0; b < cb; b += kWarp) sum += look(a, b + lane);
        if (cb > 0) {
#pragma unroll
            for (int o = kWarp / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        chunk(a, lane);
        before = (int)sum;
        // (more than 2^31 tiles: offsets that go back and forth over the same rows, and are reported; nothing is taken)
        sum += __shfl_sync(0xffffffffu, inc, 31);
        total = sum > 0x7fffffff ? 0 : (int)sum;
        if (bits) atomicOr(&g_status, bits);
    }
    // The number of tile `want` (0 <= want < total) inside this lane's sequence, or -1 if another lane has it.
    __device__ __forceinline__ int tile(const AttnArgs& a, int want, int lane) {
        while (want < before) {
            cb -= kWarp;
            chunk(a, lane);
            before -= __shfl_sync(0xffffffffu, inc, 31);
        }
        for (int here; want - before >= (here = __shfl_sync(0xffffffffu, inc, 31));) {
            cb += kWarp;
            chunk(a, lane);
            before += here;
        }
        const int at = want - before - (inc - own);
        return at >= 0 && at < own ? at : -1;
    }
};

// The next CTA of the grid that has not started is taken over (asynchronously; 16 bytes at `dst`, counted
// on `bar`), and what came of it.
__device__ __forceinline__ void steal_block(uint32_t dst, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool stolen_block(uint32_t src, uint32_t* block) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}\n"
        : "=r"(ok), "=r"(x)
        : "r"(src)
        : "memory");
    *block = x;
    return ok != 0;
}

// PG: keys and values in the pages of a cache
template <int D, int NT, bool PG>
__global__ void __launch_bounds__((NT + 1) * 128, 3 - NT) attn_tc_kernel(const __grid_constant__ Maps maps, const AttnArgs a) {
    using C = Cfg<D, NT>;
    constexpr int kMmaWarp = C::kMmaWarp, kCap = C::kCap;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    enum {
        B_ITEM = 0, B_ITEMFREE = 2, B_STEAL = 4, B_LOADED = 5, B_Q = 6, B_QFREE = B_Q + NT, B_S = B_QFREE + NT, B_P = B_S + NT, B_O = B_P + NT,
        B_DONE = B_O + NT, B_FULL, B_EMPTY = B_FULL + kCap, B_ARMED = B_EMPTY + kCap, B_CLEAN = B_ARMED + kClean,
        B_N = B_CLEAN + kClean
    };
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ __align__(16) uint4 stolen;
    __shared__ Item items[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sm, odd_sm[2];
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.q)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_ITEM + i), 1);
            mbar_init(bar(B_ITEMFREE + i), 4 * NT + 3);     // softmax warps, MMA, loader, cleaner
        }
        mbar_init(bar(B_STEAL), 1);
        mbar_init(bar(B_LOADED), 1);
        for (int i = 0; i < NT; ++i) {
            mbar_init(bar(B_Q + i), 1);
            mbar_init(bar(B_QFREE + i), 1);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4);
            mbar_init(bar(B_O + i), 1);
        }
        mbar_init(bar(B_DONE), 1);
        for (int s = 0; s < kCap; ++s) {
            mbar_init(bar(B_FULL + s), 1);
            mbar_init(bar(B_EMPTY + s), 1);
        }
        for (int s = 0; s < kClean; ++s) {
            mbar_init(bar(B_ARMED + s), 1);
            mbar_init(bar(B_CLEAN + s), 1);
        }
        abort_sm = 0;
    }
    if (warp == kMmaWarp) tmem_alloc<C::kTmem>(smem_u32(&tmem_base));
    wait_for_last_kernel();
    Finder<C::kQ, PG> find;
    // (before the barriers are there, as nothing of it needs them: five short prompts 11.2 -> 10.4 us; with two
    // tiles it costs the softmax registers, 4 x 4096 x 32 heads 415 -> 431 us)
    if (NT == 1 && warp == C::kItemWarp) find.start(a, lane);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tb = tmem_base;

    auto wait_for = [&](int i, uint32_t parity, uint64_t limit) -> bool {
        const uint32_t x = bar(i);
        uint64_t start = 0;
        for (int it = 0;; ++it) {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}\n"
                : "=r"(ok)
                : "r"(x), "r"(parity)
                : "memory");
            if (ok) return true;
            if (*reinterpret_cast<volatile int*>(&abort_sm)) return false;
            const uint64_t now = globaltimer_ns();
            if (it == 0) start = now;
            else if (now - start > limit) {
                abort_sm = 1;
                return false;
            }
        }
    };
    auto wait = [&](int i, uint32_t parity) -> bool { return wait_for(i, parity, kWaitNs); };
    // Every role walks the same items: item n is in slot n & 1; `last` of them has live = 0.
    auto get_item = [&](int n, Item* t) -> bool {
        if (!wait_for(B_ITEM + (n & 1), (uint32_t)(n >> 1) & 1u, kItemNs)) return false;
        *t = items[n & 1];
        return t->live != 0;
    };
    // Pairs, counted over all items: pair P is what the products of one turn read, V of a block and K of
    // the block behind it (an item's first pair: only K; its last: only V).  It has one barrier for
    // "loaded", one for "read" and one place in the ring, P % kCap of each, so that it is loaded when pair
    // P - kCap has been read.
    auto full_of = [&](int P) { return B_FULL + P % kCap; };
    auto empty_of = [&](int P) { return B_EMPTY + P % kCap; };
    auto phase = [&](int P) { return (uint32_t)(P / kCap) & 1u; };
    auto v_of = [&](int P) { return (uint32_t)(NT + 2 * (P % kCap)) * C::kTileBytes; };       // offset of its V
    auto k_of = [&](int P) { return (uint32_t)(NT + 2 * (P % kCap) + 1) * C::kTileBytes; };   // ... of its K

    if (warp >= kMmaWarp) {
        // (what the block was launched with, 168 or 128 a thread, given out anew)
        if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == C::kItemWarp) {
            // ================================ items ================================
            // This CTA's own block first, then blocks of the grid that have not started, one ahead of the
            // work: none looks tiles up or loads its first tiles while the tensor core waits.
            if (NT == 2) find.start(a, lane);
            bool ok = true, more = true;
            uint32_t block = blockIdx.x;
            int n = 0, steals = 0;
            while (ok && more) {
                const unsigned u = block / (unsigned)a.Hq;
                if (u < (unsigned)find.total) {
                    const int at = find.tile(a, find.total - 1 - (int)u, lane);
                    if (n >= 2) ok = __all_sync(0xffffffffu, wait_for(B_ITEMFREE + (n & 1), (uint32_t)(n / 2 - 1) & 1u, kItemNs));
                    if (!ok) break;
                    if (at >= 0) {
                        Item& t = items[n & 1];
                        t.b = find.cb + lane;
                        t.q0 = find.q0;
                        t.lq = find.lq;
                        t.k0 = find.k0;
                        t.lk = find.lk;
                        t.r0 = at * C::kQ;
                        t.h = (int)(block - u * (unsigned)a.Hq);
                        t.live = 1;
                        odd_sm[n & 1] = 0;
                        mbar_arrive1(bar(B_ITEM + (n & 1)));
                    }
                    __syncwarp();
                    ++n;
                    // the next block is taken when this one's last load is under way, and not before: an
                    // item that waits for a CTA busy with long ones would be missed elsewhere at the end
                    ok = __all_sync(0xffffffffu, wait_for(B_LOADED, (uint32_t)(n - 1) & 1u, kItemNs));
                    if (!ok) break;
                }
                if (lane == 0) {
                    mbar_expect(bar(B_STEAL), 16);
                    steal_block(smem_u32(&stolen), bar(B_STEAL));
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, wait(B_STEAL, (uint32_t)steals & 1u));
                if (!ok) mbar_wait(bar(B_STEAL), (uint32_t)steals & 1u, kWaitNs);   // (given up elsewhere: the answer is still to come)
                ++steals;
                if (ok) more = stolen_block(smem_u32(&stolen), &block);
                fence_async_smem();                                    // (read before the next answer lands there)
                __syncwarp();
            }
            // the end: an item that is none
            if (ok && n >= 2) ok = __all_sync(0xffffffffu, wait_for(B_ITEMFREE + (n & 1), (uint32_t)(n / 2 - 1) & 1u, kItemNs));
            if (ok && lane == 0) {
                items[n & 1].live = 0;
                mbar_arrive1(bar(B_ITEM + (n & 1)));
            }
        } else if (warp == C::kLoadWarp) {
            // ================================ loader ================================
            // One thread; with pages the whole warp: a lane looks up and loads one box (of up to 128 rows of a
            // page, 64 channels) of a pair.  Tokens behind the sequence and pages outside the cache are read
            // behind the pool's end, as zeros.
            if (PG || lane == 0) {
                auto agree = [&](bool x) -> bool {
                    if constexpr (PG) return __all_sync(0xffffffffu, x);
                    else return x;
                };
                [[maybe_unused]] const int part = lane >> 4, bx = (lane >> 3) & 1;         // K or V, 64 channels
                [[maybe_unused]] const int rows = PG ? min(a.p.page, kN) : kN, by = (lane & 7) * rows;
                [[maybe_unused]] bool bad = false;
                Item t;
                bool ok = true;
                int P = 0, cleans = 0, nq[NT] = {};
                for (int n = 0; ok && agree(get_item(n, &t)); ++n) {
                    const Span<NT> sp(t);
                    const int hk = t.h / a.G;
                    auto load_q = [&](int i) {
                        if (sp.nb[i] == 0) return;
                        if (nq[i] > 0 && !(ok = agree(wait(B_QFREE + i, (uint32_t)(nq[i] - 1) & 1u)))) return;
                        ++nq[i];
                        if (PG && lane > 0) return;
                        mbar_expect(bar(B_Q + i), C::kTileBytes);
                        for (int x = 0; x < D / 64; ++x)
                            tma_load3(sb + (uint32_t)i * C::kTileBytes + 16384u * x, &maps.q, 64 * x, t.h, t.q0 + t.r0 + kM * i, bar(B_Q + i));
                    };
                    if (sp.nmax > 0) {
                        load_q(0);
                        const bool give_up = gives_up(a.give_up, P, sp.nmax + 1);
                        const int stop = give_up ? a.give_up - P : sp.nmax + 1;
                        for (int p = 0; p < stop && ok; ++p) {
                            [[maybe_unused]] int pos = 0, entry = 0;
                            [[maybe_unused]] bool mine = false;
                            if constexpr (PG) {
                                // (looked up before the wait)
                                mine = bx < D / 64 && by < kN && (part ? p > 0 : p < sp.nmax);
                                pos = (p - part) * kN + by;
                                const bool in = mine && pos < t.lk;
                                const int page = in ? paged_page(a.p, t.b, pos) : -1;
                                bad |= in && page < 0;
                                entry = (page < 0 ? a.p.n_pages : page) * a.p.Hkv + (page < 0 ? 0 : hk);
                            }
                            if (P >= kCap && !(ok = agree(wait(empty_of(P), phase(P - kCap))))) break;
                            const int full = full_of(P);
                            if (!PG || lane == 0) mbar_expect(bar(full), (uint32_t)((p > 0) + (p < sp.nmax)) * C::kTileBytes);
                            if constexpr (PG) {
                                __syncwarp();
                                if (mine)
                                    tma_load4(sb + (part ? v_of(P) : k_of(P)) + 16384u * bx + 128u * by, part ? &maps.v : &maps.k, 0,
                                              pos & (a.p.page - 1), bx, entry, bar(full));
                            } else {
                                if (p > 0)
                                    for (int x = 0; x < D / 64; ++x)
                                        tma_load3(sb + v_of(P) + 16384u * x, &maps.v, 64 * x, hk, t.k0 + (p - 1) * kN, bar(full));
                                if (p < sp.nmax)
                                    for (int x = 0; x < D / 64; ++x)
                                        tma_load3(sb + k_of(P) + 16384u * x, &maps.k, 64 * x, hk, t.k0 + p * kN, bar(full));
                            }
                            if (p > sp.nf && (!PG || lane == 0)) mbar_arrive1(bar(B_ARMED + cleans % kClean));
                            cleans += p > sp.nf;
                            ++P;
                            if (p == 0 && NT == 2) load_q(NT - 1);
                        }
                        if (give_up) {
                            abort_sm = 1;
                            ok = false;
                        }
                    }
                    if (PG) __syncwarp();                              // (every lane has read the item)
                    if (ok && (!PG || lane == 0)) {
                        mbar_arrive1(bar(B_LOADED));
                        mbar_arrive1(bar(B_ITEMFREE + (n & 1)));
                    }
                }
                // leave no copy in flight
                for (int x = max(0, P - kCap); x < P; ++x) mbar_wait(bar(full_of(x)), phase(x), kWaitNs);
                for (int i = 0; i < NT; ++i)
                    if (nq[i] > 0) mbar_wait(bar(B_Q + i), (uint32_t)(nq[i] - 1) & 1u, kWaitNs);
                if (PG && bad) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
            }
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // ================================ MMA issue ================================
            if (lane == 0) {
                constexpr uint32_t id_s = idesc_bf16(kM, kN, 0), id_o = idesc_bf16(kM, D, 1);
                constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
                Item t;
                bool ok = true;
                int P = 0, cleans = 0, nq[NT] = {}, ns[NT] = {};      // Q tiles, blocks of the tile before this item
                for (int n = 0; ok && get_item(n, &t); ++n) {
                    const Span<NT> sp(t);
                    // S_i of block j (K in pair P0 + j); behind the item's last one Q_i may be overwritten
                    auto s_mma = [&](int i, int j, int pk) {
                        const uint32_t q = desc_lo(sb + (uint32_t)i * C::kTileBytes, 16), k = desc_lo(sb + k_of(pk), 16);
#pragma unroll
                        for (int x = 0; x < D / 16; ++x) {
                            const uint32_t o = (uint32_t)(x >> 2) * 1024u + (uint32_t)(x & 3) * 2u;   // 16-byte units
                            mma_ss(tb + C::TS(i), q + o, k + o, hi, id_s, x > 0);
                        }
                        mma_commit(bar(B_S + i));
                        if (j + 1 == sp.nb[i]) mma_commit(bar(B_QFREE + i));
                    };
                    if (sp.nmax > 0) {
                        ok = wait(full_of(P), phase(P));
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            if (ok && sp.nb[i] > 0) {
                                ok = wait(B_Q + i, (uint32_t)nq[i]++ & 1u);
                                fence_after();
                                if (ok) s_mma(i, 0, P);
                            }
                        mma_commit(bar(empty_of(P)));
                        ++P;
                        for (int j = 0; j < sp.nmax && ok; ++j, ++P) {
                            // V of block j and K of block j + 1
                            ok = wait(full_of(P), phase(P));
                            if (ok && j >= sp.nf) {
                                ok = wait(B_CLEAN + cleans % kClean, (uint32_t)(cleans / kClean) & 1u);
                                ++cleans;
                            }
                            const uint32_t v = desc_lo(sb + v_of(P), 16384);
#pragma unroll
                            for (int i = 0; i < NT; ++i) {
                                if (ok && j < sp.nb[i]) {
                                    if (!(ok = wait(B_P + i, (uint32_t)(ns[i] + j) & 1u))) break;
                                    fence_after();
#pragma unroll
                                    for (int x = 0; x < kN / 16; ++x)
                                        mma_ts(tb + C::TO(i), tb + C::TS(i) + 8 * x, v + 128u * x, hi, id_o, x > 0 ? 1u : (uint32_t)j);
                                    if (j + 1 < sp.nb[i]) s_mma(i, j + 1, P);
                                    else mma_commit(bar(B_O + i));
                                }
                            }
                            mma_commit(bar(empty_of(P)));
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i) ns[i] += sp.nb[i];
                    }
                    if (ok) mbar_arrive1(bar(B_ITEMFREE + (n & 1)));
                }
                // leave no product in flight
                mma_commit(bar(B_DONE));
                if (!mbar_wait(bar(B_DONE), 0, kWaitNs)) abort_sm = 1;
            }
            __syncwarp();
        } else {
            // ================================ cleaner ================================
            Item t;
            int P = 0, cleans = 0;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                if (!__all_sync(0xffffffffu, get_item(n, &t))) break;
                const Span<NT> sp(t);
                for (int j = sp.nf; j < sp.nmax && ok; ++j, ++cleans) {
                    // (a pair's "loaded" can be told from the one before at its place only once it is armed)
                    const int pv = P + j + 1, c = cleans % kClean;
                    const uint32_t par = (uint32_t)(cleans / kClean) & 1u;
                    ok = wait_for(B_ARMED + c, par, kItemNs) && wait(full_of(pv), phase(pv));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int valid = min(kN, t.lk - j * kN);
                    // 16-byte chunks in memory order, eight (32 rows of 64 channels) in flight.  Nearly always all are
                    // finite: the largest magnitude tells, one instruction a word (a test of every word's exponents, three,
                    // took 4 x 4096 x 32 heads 412 us, now 382, and 16 prompts of 512 tokens 76, now 67).
                    uint4* p = reinterpret_cast<uint4*>(sm + v_of(pv)) + lane;
                    uint32_t top[4] = {0u, 0u, 0u, 0u};
                    auto look = [&](const uint4& y) {
                        top[0] = max_abs2(top[0], y.x);
                        top[1] = max_abs2(top[1], y.y);
                        top[2] = max_abs2(top[2], y.z);
                        top[3] = max_abs2(top[3], y.w);
                    };
                    if (valid == kN) {
#pragma unroll 1
                        for (int x0 = 0; x0 < kN * D / 8 / 32; x0 += 8) {
                            uint4 y[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) y[x] = p[32 * (x0 + x)];
#pragma unroll
                            for (int x = 0; x < 8; ++x) look(y[x]);
                        }
                    } else {
#pragma unroll 1
                        for (int x0 = 0; x0 < kN * D / 8 / 32; x0 += 8) {
                            const int left = valid - ((4 * x0) & (kN - 1)), row = lane >> 3;   // (4 x + lane / 8 of the 32)
                            if (left > 0) {
                                uint4 y[8];
#pragma unroll
                                for (int x = 0; x < 8; ++x) y[x] = p[32 * (x0 + x)];
#pragma unroll
                                for (int x = 0; x < 8; ++x)
                                    if (4 * x + row < left) look(y[x]);
                            }
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                if (4 * x + row >= left) p[32 * (x0 + x)] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    const uint32_t most = max_abs2(max_abs2(top[0], top[1]), max_abs2(top[2], top[3]));
                    if (__any_sync(0xffffffffu, (most & 0x7f80u) == 0x7f80u || (most & 0x7f800000u) == 0x7f800000u)) {
                        if (lane == 0) *reinterpret_cast<volatile int*>(&odd_sm[n & 1]) = 1;
#pragma unroll 1
                        for (int x = 0; x < kN * D / 8 / 32; ++x) {
                            const uint4 z = p[32 * x];
                            uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const bool lo = (w[e] & 0x7f80u) == 0x7f80u, up = (w[e] & 0x7f800000u) == 0x7f800000u;
                                w[e] &= (lo ? 0xffff0000u : ~0u) & (up ? 0xffffu : ~0u);
                            }
                            p[32 * x] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    fence_async_smem();
                    __threadfence_block();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(bar(B_CLEAN + c));
                }
                if (sp.nmax > 0) P += sp.nmax + 1;
                if (ok && lane == 0) mbar_arrive1(bar(B_ITEMFREE + (n & 1)));
            }
        }
    } else {
        // ================================ softmax ================================
        if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;                    // tile, row of the tile
        const uint32_t lo = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tb + lo + C::TS(i), to = tb + lo + C::TO(i);
        const float c = a.scale_log2;
        uint8_t* stage = sm + (size_t)(NT + 2 * kCap) * C::kTileBytes + (size_t)i * C::kStageBytes;
        int ns = 0, no = 0;                                                     // blocks, items with blocks so far
        for (int it = 0;; ++it) {
            Item t;
            if (!__all_sync(0xffffffffu, get_item(it, &t))) break;
            const Span<NT> sp(t);
            const int row = t.r0 + kM * i + r, shift = t.lk - t.lq, n = sp.nb[i];   // (the row may lie behind the sequence)
            const int last = min(row + shift, t.lk - 1);                            // the row's last key
            const int wfull = max(0, min(t.lk, row - lane + shift + 1)) / kN;       // blocks the warp's rows see whole
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < n && ok; ++j) {
                if (!(ok = __all_sync(0xffffffffu, wait(B_S + i, (uint32_t)(ns + j) & 1u)))) break;
                fence_after();
                float s[kN];
#pragma unroll
                for (int x = 0; x < kN; x += 32) tmem_ld32(ts + x, s + x);
                tmem_wait_ld();
                if (j >= wfull) {
                    // 32 columns at a time: most are seen whole by the warp's rows even here
                    const int lim = last - j * kN, w0 = __reduce_min_sync(0xffffffffu, lim);
#pragma unroll
                    for (int x = 0; x < kN; x += 32) {
                        if (w0 >= x + 31) continue;
#pragma unroll
                        for (int y = x; y < x + 32; ++y) s[y] = y <= lim ? s[y] : -INFINITY;
                    }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int x = 4; x < kN; ++x) mx[x & 3] = fmaxf(mx[x & 3], s[x]);
                const float top = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), c, kRaise);
                const bool need = top > m + kRaise;
                if (j == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, need)) {
                    // (O_i is quiet: S of this block was issued behind the block before's P V, and is done)
                    const float f = need ? ex2(m - top) : 1.f;
                    l *= f;
                    // (rare, and with S in registers: 16 columns at a time)
#pragma unroll 1
                    for (int x = 0; x < D; x += 16) {
                        uint32_t o[16];
                        tmem_ld16(to + x, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                        tmem_st16(to + x, o);
                    }
                    if (need) m = top;
                }
                const float base = m == -INFINITY ? 0.f : m;
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
#pragma unroll
                for (int x = 0; x < kN; x += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        float2 e = fma2(make_float2(s[x + 2 * y], s[x + 2 * y + 1]), c2, b2);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        ls[y & 1] = add2(ls[y & 1], e);
                        const __nv_bfloat162 bp = __floats2bfloat162_rn(e.x, e.y);
                        p[y] = *reinterpret_cast<const uint32_t*>(&bp);
                    }
                    tmem_st16(ts + x / 2, p);
                }
                l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bar(B_P + i));
            }
            // ---- o = O / l ----
            if (n > 0 && ok) ok = __all_sync(0xffffffffu, wait(B_O + i, (uint32_t)no & 1u));
            if (!ok) break;
            fence_after();
            ns += n;
            no += n > 0;
            const bool none = last < 0 || n == 0;
            const float inv = 1.f / l;
            const bool odd = *reinterpret_cast<volatile int*>(&odd_sm[it & 1]) != 0;
            const int rest = t.lq - (row - lane);                   // rows of the warp inside the sequence
            __nv_bfloat16* O = reinterpret_cast<__nv_bfloat16*>(a.O.data) + (int64_t)(t.q0 + row - lane) * a.O.row + (int64_t)t.h * a.O.head;
            // 32 columns at a time through shared memory (64-byte rows, 16-byte chunks swizzled), so that
            // whole sectors go out
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(to + x, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = none ? 0.f : o[y] * inv;
                if (odd && lane < rest) {
                    // values that are not finite and were kept out of the products: for the keys the row sees
#pragma unroll 1
                    for (int key = sp.nf * kN; key <= last; ++key) {
                        int64_t at;
                        if constexpr (PG) {
                            const int page = paged_page(a.p, t.b, key);
                            if (page < 0) continue;
                            at = paged_offset(a.p, page, t.h / a.G, key);
                        } else {
                            at = (int64_t)(t.k0 + key) * a.V.row + (int64_t)(t.h / a.G) * a.V.head;
                        }
                        const __nv_bfloat16* V = reinterpret_cast<const __nv_bfloat16*>(PG ? a.p.V : a.V.data) + at + x;
#pragma unroll
                        for (int y = 0; y < 32; ++y) {
                            const float v = __bfloat162float(V[y]);
                            if (!(fabsf(v) <= 3.4e38f)) o[y] += v;
                        }
                    }
                }
                uint32_t p[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    const __nv_bfloat162 bp = __floats2bfloat162_rn(o[2 * y], o[2 * y + 1]);
                    p[y] = *reinterpret_cast<const uint32_t*>(&bp);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<uint4*>(stage + r * 64 + ((y ^ (r >> 1)) & 3) * 16) = make_uint4(p[4 * y], p[4 * y + 1], p[4 * y + 2], p[4 * y + 3]);
                __syncwarp();
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int rr = 8 * y + (lane >> 2), wr = (warp & 3) * 32 + rr;
                    const uint4 z = *reinterpret_cast<const uint4*>(stage + wr * 64 + (((lane & 3) ^ (wr >> 1)) & 3) * 16);
                    if (rr < rest) *reinterpret_cast<uint4*>(O + (int64_t)rr * a.O.row + x + 8 * (lane & 3)) = z;
                }
                __syncwarp();
            }
            if (a.lse && lane < rest)
                a.lse[(int64_t)t.h * a.total_q + t.q0 + row] = none ? -INFINITY : (m + log2f(l)) * kAttnLn2;
            // (O_i and odd_sm are read: the next item's products wait for this warp's next weights)
            fence_before();
            if (lane == 0) mbar_arrive1(bar(B_ITEMFREE + (it & 1)));
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (abort_sm && tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
    if (warp == kMmaWarp) tmem_dealloc<C::kTmem>(tb);
}

bool make_map(CUtensorMap* m, const Rows& r, int64_t rows, int heads, int d) {
    return make_tmap_rows(m, r.data, rows, heads, d, r.row, r.head, kM);
}

template <int D, int NT, bool PG>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
    using C = Cfg<D, NT>;
    Maps maps;
    const int Hkv = a.Hq / a.G;
    const int64_t rows_k = a.total_k > 0 ? a.total_k : 1;
    auto keys_map = [&](CUtensorMap* m, const Rows& r, const char* pool) {
        if (!PG) return make_map(m, r, rows_k, Hkv, D);
        return make_tmap_pages(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, D, a.p.page, (int64_t)a.p.n_pages * Hkv, a.p.page < kN ? a.p.page : kN, 1);
    };
    if (!make_map(&maps.q, a.Q, a.total_q, a.Hq, D) || !keys_map(&maps.k, a.K, a.p.K) || !keys_map(&maps.v, a.V, a.p.V))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_smem(attn_tc_kernel<D, NT, PG>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    // at most this many tiles for any cut of total_q rows into n_seq sequences
    const int64_t tiles = ((int64_t)a.total_q + (int64_t)a.n_seq * (C::kQ - 1)) / C::kQ;
    return launch_behind(attn_tc_kernel<D, NT, PG>, (unsigned)(tiles * a.Hq), C::kThreads, C::kSmem, st, maps, a);
}

}  // namespace

// One or two tiles per CTA?  An item costs about o + s B microseconds, B the key blocks its tiles read on
// average: measured on prompts of 128 to 8192 tokens, 8 heads (us; two tiles: a round of 152 CTAs, one
// tile: a round of 304, two on an SM),
//            d = 128, two: 6.8 + 1.39 B   one: 6.4 + 1.67 B      d = 64, two: 5.2 + 1.18 B   one: 5.0 + 1.30 B
// so two tiles for long sequences (19 prompts of 4096 tokens, d = 128: 469 against 537 us), and one for short
// ones (304 of 128 tokens: 61 against 79 us) and where its finer cut saves a round (10 tiles of ~50 blocks,
// 16 heads, d = 64: 80 against 121 us).  The tiles of a ragged batch are not known here: for each sequence half a
// tile is added, less with two (their last item has one tile half of the time), or, where the rounds are few and
// a tile more can cost a whole one, what the grid may come to.
static bool one_tile(const AttnArgs& a) {
    const double n = a.n_seq, lq = a.total_q / n, lk = a.total_k / n;
    const double blocks = (lk > lq ? lk - lq / 2 : lk / 2) / kN + 0.5;
    auto cost = [&](int nt, double o, double s) {
        const double q = nt * kM, slots = nt == 2 ? 152 : 304;
        const double most = (double)(((int64_t)a.total_q + (int64_t)a.n_seq * (int64_t)(q - 1)) / (int64_t)q) * a.Hq / slots;
        const double mean = (a.total_q / q + (nt == 2 ? 0.3 : 0.5) * n) * a.Hq / slots;
        return (most <= 4 ? std::ceil(most) : mean) * (o + s * blocks);
    };
    return a.d == 128 ? cost(1, 6.4, 1.67) < cost(2, 6.8, 1.39) : cost(1, 5.0, 1.30) < cost(2, 5.2, 1.18);
}

template <bool PG> static cudaError_t launch_form(const AttnArgs& a, cudaStream_t st) {
    const bool one = one_tile(a);
    if (a.d == 128) return one ? launch<128, 1, PG>(a, st) : launch<128, 2, PG>(a, st);
    return one ? launch<64, 1, PG>(a, st) : launch<64, 2, PG>(a, st);
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st) {
    return a.p.table ? launch_form<true>(a, st) : launch_form<false>(a, st);
}

cudaError_t attn_tc_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
