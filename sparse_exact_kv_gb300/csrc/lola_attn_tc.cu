// K8 (bf16, tensor cores): causal softmax attention over packed prompts.
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j <= i + Lk - Lq.  One pass over
// the keys in blocks of 128 with a running maximum m and sum l per row (log2 units):
//   S = Q K^T,  P = 2^{c S - m},  l += sum P,  O += P V,      o = O / l,
// m is raised lazily: O and l are rescaled (in TMEM) only when a block's maximum passes m by more
// than 2^8, so that P and l stay far inside float32 and bfloat16, and blocks rarely wait for O.
//
// A CTA takes 256 queries of one head as two tiles of 128 (MMA M = 128, TMEM lane = query) that share
// every K and V block; while the tensor core works for one tile, the other tile's softmax runs.  Short
// sequences take one tile per CTA and two CTAs per SM instead, each in half an SM (see one_tile below).
// Warps (of two tiles):
//   * 9 (loader): Q, K and V tiles by TMA, 128-byte swizzle, into a ring of K and V blocks;
//   * 8 (MMA, one thread): per block and tile O_i += P_i V_j, then S_i = Q_i K_{j+1}^T.  P_i
//     (bf16, read from TMEM as the A operand) lies over S_i's columns: the products of one thread
//     run in order, so S_i of the next block cannot overtake the read of P_i;
//   * 0-3, 4-7 (softmax of tile 0, 1; one thread per query): the row of S into registers,
//     mask on the blocks that some row does not see whole, maximum, weights, P into TMEM;
//   * 10-11 (cleaners): on those same blocks, V rows behind the sequence and values that are
//     not finite are zeroed in shared memory before the product (0 x NaN would reach rows
//     that do not see them); the values taken out are added back in the epilogue, for the rows
//     that see them.
// What bounds it: for long sequences the tensor core and its power (16 heads of 32768 tokens, d = 128:
// 2.96 ms, 1483 TFLOP/s of the measured 1849); a block pair's products take about 2300 cycles of the
// issuing thread's 2900-3200, the rest is its wait for the weights (a softmax is 1100 cycles, behind it
// the other tile's products).  For short ones the start and end of a CTA: about 2200 cycles of tile
// lookup, 3500 until the first scores, 2500 of epilogue.
// Tried and slower: releasing P in halves, comparing S by column groups while it loads, one MMA thread
// for each tile (their products interleave: 3.20 ms), the next pair's waits between the products.
// Every wait is bounded (1 s, then LOLA_ATTN_TIMEOUT).
#include <cuda.h>

#include <cmath>

#include "lola_attn.cuh"
#include "lola_tc.cuh"

namespace lola {
namespace {

using namespace tc;

__device__ int32_t g_status;

constexpr int kM = 128;                  // queries per tile
constexpr int kN = 128;                  // keys per block
constexpr int kPairs = 4;                // barriers of the pairs (see the kernel)
constexpr float kRaise = 8.0f;           // m is raised when a block's maximum passes it by this (log2)
constexpr uint64_t kWaitNs = 1000000000ull;

// NT: query tiles of a CTA.  Two: one CTA per SM, K and V blocks shared by 256 queries.  One: two CTAs
// per SM, each with its own ring (half the shared memory, half of TMEM).
template <int D, int NT> struct Cfg {
    static constexpr int kQ = NT * kM;                     // queries per CTA
    static constexpr int kThreads = (NT + 1) * 128;
    static constexpr int kMmaWarp = 4 * NT, kLoadWarp = kMmaWarp + 1, kCleanWarp0 = kMmaWarp + 2;
    static constexpr int kTileBytes = kM * D * 2;          // a Q tile, a K block or a V block
    static constexpr int kStages = NT == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 2 : 5);   // K and V blocks in the ring
    static constexpr int kSmem = (NT + kStages) * kTileBytes + 1024;
    static constexpr int kTmem = 256 * NT;                 // columns
    __device__ static constexpr uint32_t TS(int i) { return 128u * i; }            // S (P over its first half)
    __device__ static constexpr uint32_t TO(int i) { return 128u * NT + (uint32_t)D * i; }
};

struct Maps {
    CUtensorMap q, k, v;   // [rows][heads][d], boxes of 128 rows x 1 head x 64 channels
};


__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Products whose shared-memory descriptors come as a low word (address and leading offset in 16-byte
// units) and a high word that all of them share (stride 1024, version, swizzle): one thread issues 32 of
// them a block, and building the 64-bit descriptors each time took longer than the products.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma_ss(uint32_t tmem, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}\n" ::"r"(tmem),
        "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t tmem, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}\n" ::"r"(tmem),
        "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc));
}
// 16 consecutive 32-bit columns of this thread's TMEM lane (warp-collective)
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// two float32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t x, y, z, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t x, y, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}

template <int D, int NT>
__global__ void __launch_bounds__((NT + 1) * 128, 3 - NT) attn_tc_kernel(const __grid_constant__ Maps maps, const AttnArgs a) {
    using C = Cfg<D, NT>;
    constexpr int kMmaWarp = C::kMmaWarp, kLoadWarp = C::kLoadWarp, kCleanWarp0 = C::kCleanWarp0, kQ = C::kQ;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    enum {
        B_Q = 0, B_S = 2, B_P = 4, B_O = 6, B_DONE = 8, B_FULL = 9, B_EMPTY = B_FULL + kPairs, B_CLEAN = B_EMPTY + kPairs,
        B_ARMED = B_CLEAN + kPairs, B_N = B_ARMED + kPairs
    };
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sm, odd_sm;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.q)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
        for (int i = 0; i < NT; ++i) {
            mbar_init(bar(B_Q + i), 1);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4);
            mbar_init(bar(B_O + i), 1);
        }
        mbar_init(bar(B_DONE), 1);
        for (int s = 0; s < kPairs; ++s) {
            mbar_init(bar(B_CLEAN + s), 2);
            mbar_init(bar(B_ARMED + s), 1);
            mbar_init(bar(B_FULL + s), 1);
            mbar_init(bar(B_EMPTY + s), 1);
        }
        abort_sm = 0;
        odd_sm = 0;
    }
    if (warp == kMmaWarp) tmem_alloc<C::kTmem>(smem_u32(&tmem_base));
    const int h = blockIdx.x % (unsigned)a.Hq;
    TilePos at;
    const bool live = find_tile<C::kThreads, kQ>(a, (int)(blockIdx.x / (unsigned)a.Hq), &at);
    if (at.bad) atomicOr(&g_status, (int)LOLA_ATTN_BAD_OFFSETS);
    if (!live) {
        if (warp == kMmaWarp) {
            __syncwarp();
            tmem_dealloc<C::kTmem>(*reinterpret_cast<volatile uint32_t*>(&tmem_base));
        }
        return;
    }
    const int q0 = at.q0, lq = at.lq, k0 = at.k0, lk = at.lk, r0 = at.tile * kQ, shift = lk - lq;
    // blocks that tile i reads, and those that all its rows see whole
    int nb[NT], nf = 0x7fffffff, nmax = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int first = r0 + kM * i, last = min(first + kM, lq) - 1;      // the tile's rows
        nb[i] = first < lq ? (max(0, min(lk, last + shift + 1)) + kN - 1) / kN : 0;
        if (nb[i] > 0) nf = min(nf, max(0, min(lk, first + shift + 1)) / kN);
        nmax = max(nmax, nb[i]);
    }

    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tb = tmem_base;

    auto wait = [&](int i, uint32_t parity) -> bool {
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
            else if (now - start > kWaitNs) {
                abort_sm = 1;
                return false;
            }
        }
    };
    // Ring: block j's K is load 2 j, its V load 2 j + 1.  Pair p is what the products of one turn read, V of
    // block p - 1 and K of block p (pair 0: only K): it has one barrier for "loaded" and one for "read",
    // p % 4 of either, so a pair is loaded only when the one four before it has been read.
    auto stage = [&](int x) { return x % C::kStages; };
    auto pair = [&](int p) { return p & (kPairs - 1); };
    auto phase = [&](int p) { return (uint32_t)(p / kPairs) & 1u; };
    auto ring = [&](int x) { return sb + (uint32_t)(NT + stage(x)) * C::kTileBytes; };

    if (warp >= kMmaWarp) {
        // (what the block was launched with, 168 or 128 a thread, given out anew)
        if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == kLoadWarp) {
            // ================================ loader ================================
            if (lane == 0 && nmax > 0) {
                const int hk = h / a.G;
                auto load = [&](const CUtensorMap* m, int row, int head, uint32_t dst, int bi) {
                    mbar_expect(bar(bi), C::kTileBytes);
                    for (int x = 0; x < D / 64; ++x) tma_load3(dst + 16384u * x, m, 64 * x, head, row, bar(bi));
                };
                if (nb[0] > 0) load(&maps.q, q0 + r0, h, sb, B_Q);
                bool ok = true;
                int p = 0, waited = 0;
                for (; p <= nmax && ok; ++p) {
                    const int last = p < nmax ? 2 * p : 2 * p - 1;              // the pair's last load
                    // what its stages and its barriers held before has been read
                    const int held = last >= C::kStages ? (last - C::kStages + 1) / 2 : -1;
                    while (ok && waited <= max(held, p - kPairs)) {
                        ok = wait(B_EMPTY + pair(waited), phase(waited));
                        ++waited;
                    }
                    if (!ok) break;
                    const int full = B_FULL + pair(p);
                    mbar_expect(bar(full), (uint32_t)((p > 0) + (p < nmax)) * C::kTileBytes);
                    if (p > nf) mbar_arrive1(bar(B_ARMED + pair(p)));
                    for (int n = max(0, 2 * p - 1); n <= last; ++n)
                        for (int x = 0; x < D / 64; ++x)
                            tma_load3(ring(n) + 16384u * x, n & 1 ? &maps.v : &maps.k, 64 * x, hk, k0 + (n >> 1) * kN, bar(full));
                    if (NT == 2 && p == 0 && nb[NT - 1] > 0) load(&maps.q, q0 + r0 + kM, h, sb + C::kTileBytes, B_Q + 1);
                }
                // leave no copy in flight
                for (int x = max(0, p - kPairs); x < p; ++x) mbar_wait(bar(B_FULL + pair(x)), phase(x), kWaitNs);
                for (int i = 0; i < NT; ++i)
                    if (nb[i] > 0) mbar_wait(bar(B_Q + i), 0, kWaitNs);
            }
        } else if (warp == kMmaWarp) {
            // ================================ MMA issue ================================
            if (lane == 0 && nmax > 0) {
                constexpr uint32_t id_s = idesc_bf16(kM, kN, 0), id_o = idesc_bf16(kM, D, 1);
                constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
                auto s_mma = [&](int i, int j) {
                    const uint32_t q = desc_lo(sb + (uint32_t)i * C::kTileBytes, 16), k = desc_lo(ring(2 * j), 16);
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t o = (uint32_t)(x >> 2) * 1024u + (uint32_t)(x & 3) * 2u;   // 16-byte units
                        mma_ss(tb + C::TS(i), q + o, k + o, hi, id_s, x > 0);
                    }
                    mma_commit(bar(B_S + i));
                };
                bool ok = wait(B_FULL, 0);
                for (int i = 0; i < NT && ok; ++i)
                    if (nb[i] > 0) {
                        ok = wait(B_Q + i, 0);
                        fence_after();
                        if (ok) s_mma(i, 0);
                    }
                mma_commit(bar(B_EMPTY));
                for (int j = 0; j < nmax && ok; ++j) {
                    // V of block j and K of block j + 1
                    ok = wait(B_FULL + pair(j + 1), phase(j + 1));
                    if (ok && j >= nf) ok = wait(B_CLEAN + pair(j + 1), (uint32_t)((j - nf) / kPairs) & 1u);
                    const uint32_t v = desc_lo(ring(2 * j + 1), 16384);
                    for (int i = 0; i < NT && ok; ++i) {
                        if (j < nb[i]) {
                            if (!(ok = wait(B_P + i, (uint32_t)j & 1u))) break;
                            fence_after();
#pragma unroll
                            for (int x = 0; x < kN / 16; ++x)
                                mma_ts(tb + C::TO(i), tb + C::TS(i) + 8 * x, v + 128u * x, hi, id_o, x > 0 ? 1u : (uint32_t)j);
                        }
                        if (j + 1 < nb[i]) s_mma(i, j + 1);
                        else if (j + 1 == nb[i]) mma_commit(bar(B_O + i));
                    }
                    mma_commit(bar(B_EMPTY + pair(j + 1)));
                }
                // leave no product in flight
                mma_commit(bar(B_DONE));
                if (!mbar_wait(bar(B_DONE), 0, kWaitNs)) abort_sm = 1;
            }
            __syncwarp();
        } else {
            // ================================ cleaners ================================
            const int ct = tid - kCleanWarp0 * kWarp;
            bool ok = true;
            for (int j = nf; j < nmax && ok; ++j) {
                // (a pair's "loaded" can be told from the one four pairs before only once it is armed)
                ok = wait(B_ARMED + pair(j + 1), (uint32_t)((j - nf) / kPairs) & 1u) && wait(B_FULL + pair(j + 1), phase(j + 1));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t* v = sm + (size_t)(NT + stage(2 * j + 1)) * C::kTileBytes;
                const int valid = min(kN, lk - j * kN);
                // 16-byte chunks in memory order, eight in flight; a bfloat16 is not finite iff adding 1
                // to its exponent carries into the sign
                bool odd = false;
                uint4* p = reinterpret_cast<uint4*>(v) + ct;
#pragma unroll 1
                for (int x0 = 0; x0 < kN * D / 8 / 64; x0 += 8) {
                    uint4 y[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) y[x] = p[64 * (x0 + x)];
                    uint32_t hit = 0;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int row = ((ct + 64 * (x0 + x)) >> 3) & (kN - 1);
                        const uint32_t t = ((y[x].x & 0x7f807f80u) + 0x00800080u) | ((y[x].y & 0x7f807f80u) + 0x00800080u) |
                                           ((y[x].z & 0x7f807f80u) + 0x00800080u) | ((y[x].w & 0x7f807f80u) + 0x00800080u);
                        if (row < valid) hit |= t;
                        else p[64 * (x0 + x)] = make_uint4(0, 0, 0, 0);
                    }
                    if (!(hit & 0x80008000u)) continue;
                    odd = true;
#pragma unroll 1
                    for (int x = 0; x < 8; ++x) {
                        uint4* c = p + 64 * (x0 + x);
                        const uint4 z = *c;
                        uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool lo = (w[e] & 0x7f80u) == 0x7f80u, hi = (w[e] & 0x7f800000u) == 0x7f800000u;
                            w[e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
                        }
                        *c = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (odd) *reinterpret_cast<volatile int*>(&odd_sm) = 1;
                fence_async_smem();
                __threadfence_block();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bar(B_CLEAN + pair(j + 1)));
            }
        }
    } else {
        // ================================ softmax ================================
        if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int i = warp >> 2, row = r0 + kM * i + (warp & 3) * 32 + lane;    // (may lie behind the sequence)
        const uint32_t lo = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tb + lo + C::TS(i), to = tb + lo + C::TO(i);
        const int n = nb[i], last = min(row + shift, lk - 1);                   // the row's last key
        const int wfull = max(0, min(lk, (row - lane) + shift + 1)) / kN;       // blocks the warp's rows see whole
        const float c = a.scale_log2;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n && ok; ++j) {
            if (!(ok = __all_sync(0xffffffffu, wait(B_S + i, (uint32_t)j & 1u)))) break;
            fence_after();
            float s[kN];
#pragma unroll
            for (int x = 0; x < kN; x += 32) tmem_ld32(ts + x, s + x);
            tmem_wait_ld();
            if (j >= wfull) {
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
            const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            const bool need = bm > m + kRaise;
            if (j == 0) {
                m = bm;
            } else if (__any_sync(0xffffffffu, need)) {
                // (O_i is quiet: S of this block was issued behind the block before's P V, and is done)
                const float f = need ? ex2(m - bm) : 1.f;
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
                if (need) m = bm;
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
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bar(B_P + i));
            l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        }
        // ---- o = O / l ----
        if (n > 0 && ok) ok = __all_sync(0xffffffffu, wait(B_O + i, 0));
        fence_after();
        const bool none = last < 0 || n == 0, own = row < lq && ok;
        const float inv = 1.f / l;
        const bool odd = *reinterpret_cast<volatile int*>(&odd_sm) != 0;
        // the tile's Q rows have been read: their place takes o (the same swizzled layout), from where
        // whole rows go out, 512 bytes a warp and store
        uint8_t* stagep = sm + (size_t)i * C::kTileBytes;
        const int r = (warp & 3) * 32 + lane;
        // (loops, not unrolled: straight code that runs once is fetched slower than it executes)
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
            float o[32];
            if (n > 0) {
                tmem_ld32(to + x, o);
                tmem_wait_ld();
            }
            uint32_t p[16];
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = none ? 0.f : o[y] * inv;
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                const __nv_bfloat162 bp = __floats2bfloat162_rn(o[2 * y], o[2 * y + 1]);
                p[y] = *reinterpret_cast<const uint32_t*>(&bp);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *reinterpret_cast<uint4*>(stagep + (x >> 6) * 16384 + kmaj_chunk(r, ((x & 63) >> 3) + y)) =
                    make_uint4(p[4 * y], p[4 * y + 1], p[4 * y + 2], p[4 * y + 3]);
        }
        if (odd && own) {
            // values that are not finite and were kept out of the products: for the keys the row sees
            // (rare, so small code: one channel at a time)
#pragma unroll 1
            for (int x = 0; x < D; ++x) {
                const __nv_bfloat16* V = reinterpret_cast<const __nv_bfloat16*>(a.V.data) + (int64_t)(h / a.G) * a.V.head + x;
                float add = 0.f;
#pragma unroll 1
                for (int key = nf * kN; key <= last; ++key) {
                    const float v = __bfloat162float(V[(int64_t)(k0 + key) * a.V.row]);
                    if (!(fabsf(v) <= 3.4e38f)) add += v;
                }
                __nv_bfloat16* z = reinterpret_cast<__nv_bfloat16*>(stagep + (x >> 6) * 16384 + kmaj_chunk(r, (x & 63) >> 3)) + (x & 7);
                if (add != 0.f) *z = __float2bfloat16_rn(__bfloat162float(*z) + add);
            }
        }
        __syncwarp();
        constexpr int CH = D / 8, RW = 32 / CH;                 // chunks of a row, rows of a store
        __nv_bfloat16* O = reinterpret_cast<__nv_bfloat16*>(a.O.data) + (int64_t)(q0 + row - lane) * a.O.row +
                           (int64_t)h * a.O.head;
        const int rest = ok ? lq - (row - lane) : 0;            // rows of the warp inside the sequence
        const int ch = lane % CH;
#pragma unroll 4
        for (int x = 0; x < 32; x += RW) {
            const int y = x + lane / CH;
            const uint4 z = *reinterpret_cast<const uint4*>(stagep + (ch >> 3) * 16384 + kmaj_chunk((warp & 3) * 32 + y, ch & 7));
            if (y < rest) *reinterpret_cast<uint4*>(O + (int64_t)y * a.O.row + 8 * ch) = z;
        }
        if (a.lse && own)
            a.lse[(int64_t)h * a.total_q + q0 + row] = none ? -INFINITY : (m + log2f(l)) * kAttnLn2;
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

template <int D, int NT>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
    using C = Cfg<D, NT>;
    Maps maps;
    const int Hkv = a.Hq / a.G;
    const int64_t rows_k = a.total_k > 0 ? a.total_k : 1;
    if (!make_map(&maps.q, a.Q, a.total_q, a.Hq, D) || !make_map(&maps.k, a.K, rows_k, Hkv, D) ||
        !make_map(&maps.v, a.V, rows_k, Hkv, D))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_smem(attn_tc_kernel<D, NT>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    // at most this many tiles for any cut of total_q rows into n_seq sequences
    const int64_t tiles = ((int64_t)a.total_q + (int64_t)a.n_seq * (C::kQ - 1)) / C::kQ;
    attn_tc_kernel<D, NT><<<(unsigned)(tiles * a.Hq), C::kThreads, C::kSmem, st>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

// One or two tiles per CTA?  A CTA costs about o + s B microseconds, B the key blocks its tiles read on
// average: measured on prompts of 128 to 8192 tokens, 8 heads (us; two tiles: a round of 152 CTAs, one
// tile: a round of 304, two on an SM),
//            d = 128, two: 9.7 + 1.47 B   one: 8.3 + 1.94 B      d = 64, two: 8.0 + 1.19 B   one: 6.5 + 1.32 B
// so one tile for short sequences (304 of 128 tokens, d = 128: 90 against 136 us; 19 of 4096: 645 against
// 545), and where its finer cut saves a round (10 tiles of ~50 blocks, 16 heads, d = 64: 84 against
// 126 us).  The tiles of a ragged batch are not known here: half a tile is added for each sequence, or
// what the grid may come to where the rounds are few and a tile more can cost a whole one.
static bool one_tile(const AttnArgs& a) {
    const double n = a.n_seq, lq = a.total_q / n, lk = a.total_k / n;
    const double blocks = (lk > lq ? lk - lq / 2 : lk / 2) / kN + 0.5;
    auto cost = [&](int nt, double o, double s) {
        const double q = nt * kM, slots = nt == 2 ? 152 : 304;
        const double most = (double)(((int64_t)a.total_q + (int64_t)a.n_seq * (int64_t)(q - 1)) / (int64_t)q) * a.Hq / slots;
        const double mean = (a.total_q / q + 0.5 * n) * a.Hq / slots;
        return (most <= 4 ? std::ceil(most) : std::ceil(mean)) * (o + s * blocks);
    };
    return a.d == 128 ? cost(1, 8.3, 1.94) < 0.95 * cost(2, 9.7, 1.47) : cost(1, 6.5, 1.32) < 0.95 * cost(2, 8.0, 1.19);
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st) {
    const bool one = one_tile(a);
    if (a.d == 128) return one ? launch<128, 1>(a, st) : launch<128, 2>(a, st);
    return one ? launch<64, 1>(a, st) : launch<64, 2>(a, st);
}

cudaError_t attn_tc_status_take(int32_t* bits, cudaStream_t st) { return take_word(g_status, bits, st); }

}  // namespace lola
