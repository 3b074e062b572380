// K8 (bf16, tensor cores): causal softmax attention over packed prompts.
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j <= i + Lk - Lq.  One pass over
// the keys in blocks of 128 with a running maximum m and sum l per row (log2 units):
//   S = Q K^T,  P = 2^{c S - m},  l += sum P,  O += P V,      o = O / l,
// m is raised lazily: O and l are rescaled (in TMEM) only when a block's maximum passes m by more
// than 2^8, so that P and l stay far inside float32 and bfloat16, and blocks rarely wait for O.
//
// One CTA takes 256 queries of one head as two tiles of 128 (MMA M = 128, TMEM lane = query) that
// share every K and V block; while the tensor core works for one tile, the other tile's softmax runs:
//   * warp 9 (loader): Q, K and V tiles by TMA, 128-byte swizzle, into a ring of K and V blocks;
//   * warp 8 (MMA, one thread): per block and tile O_i += P_i V_j, then S_i = Q_i K_{j+1}^T.  P_i
//     (bf16, read from TMEM as the A operand) lies over S_i's columns: the products of one thread
//     run in order, so S_i of the next block cannot overtake the read of P_i;
//   * warps 0-3, 4-7 (softmax of tile 0, 1; one thread per query): the row of S into registers,
//     mask on the blocks that some row does not see whole, maximum, weights, P into TMEM;
//   * warps 10-11 (cleaners): on those same blocks, V rows behind the sequence and values that are
//     not finite are zeroed in shared memory before the product (0 x NaN would reach rows
//     that do not see them); what was finite-less is added back in the epilogue, row by row, for
//     the rows that see it.
// Every wait is bounded (1 s, then LOLA_ATTN_TIMEOUT).
#include <cuda.h>

#include "lola_attn.cuh"
#include "lola_tc.cuh"

namespace lola {
namespace {

using namespace tc;

__device__ int32_t g_status;

constexpr int kM = 128;                  // queries per tile
constexpr int kQ = 2 * kM;               // queries per CTA
constexpr int kN = 128;                  // keys per block
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCleanWarp0 = 10;
constexpr int kThreads = 384;
constexpr float kRaise = 8.0f;           // m is raised when a block's maximum passes it by this (log2)
constexpr uint64_t kWaitNs = 1000000000ull;

template <int D> struct Cfg {
    static constexpr int kTileBytes = kM * D * 2;          // a Q tile, a K block or a V block
    static constexpr int kStages = D == 128 ? 5 : 8;       // K and V blocks in the ring
    static constexpr int kCleanPeriod = kStages % 2 ? kStages : kStages / 2;   // blocks until a V uses the same stage
    static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024;
    __device__ static constexpr uint32_t TS(int i) { return 128u * i; }          // S (P over its first half)
    __device__ static constexpr uint32_t TO(int i) { return 256u + (uint32_t)D * i; }
};

struct Maps {
    CUtensorMap q, k, v;   // [rows][heads][d], boxes of 128 rows x 1 head x 64 channels
};


__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ Maps maps, const AttnArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    enum {
        B_Q = 0, B_S = 2, B_P = 4, B_O = 6, B_DONE = 8, B_FULL = 9, B_EMPTY = B_FULL + C::kStages,
        B_CLEAN = B_EMPTY + C::kStages, B_N = B_CLEAN + C::kStages
    };
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_sm, odd_sm;
    __shared__ int64_t scan[kThreads / kWarp];
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    // ---- this CTA's tile: sequences in order, read backwards, so that the CTAs that start last
    // have the first sequence's first (shortest) tiles ----
    bool bad = false;
    auto tiles = [&](int b) -> int64_t {
        int lo, len;
        seq_rows(a.cu_q, b, a.total_q, &lo, &len, &bad);
        return (len + kQ - 1) / kQ;
    };
    const int64_t total = seq_total<kThreads>(a.n_seq, tiles, scan);
    const int64_t u = (int64_t)blockIdx.x / a.Hq;
    const int h = blockIdx.x % a.Hq;
    if (bad) atomicOr(&g_status, (int)LOLA_ATTN_BAD_OFFSETS);
    if (u >= total) return;
    int b;
    int64_t rem;
    seq_find<kThreads>(a.n_seq, tiles, total - 1 - u, scan, &b, &rem);
    int q0, lq, k0, lk;
    seq_rows(a.cu_q, b, a.total_q, &q0, &lq, &bad);
    bool badk = false;
    seq_rows(a.cu_k, b, a.total_k, &k0, &lk, &badk);
    if (badk && tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_BAD_OFFSETS);
    const int r0 = (int)rem * kQ, shift = lk - lq;
    // blocks that tile i reads, and those that all its rows see whole
    int nb[2], nf = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int first = r0 + kM * i, last = min(first + kM, lq) - 1;      // the tile's rows
        nb[i] = first < lq ? (max(0, min(lk, last + shift + 1)) + kN - 1) / kN : 0;
        if (nb[i] > 0) nf = min(nf, max(0, min(lk, first + shift + 1)) / kN);
    }
    const int nmax = max(nb[0], nb[1]);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_Q + i), 1);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4);
            mbar_init(bar(B_O + i), 1);
        }
        mbar_init(bar(B_DONE), 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar(B_CLEAN + s), 2);
            mbar_init(bar(B_FULL + s), 1);
            mbar_init(bar(B_EMPTY + s), 1);
        }
        abort_sm = 0;
        odd_sm = 0;
    }
    if (warp == kMmaWarp) tmem_alloc<512>(smem_u32(&tmem_base));
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
    // ring: block j's K is load 2 j, its V load 2 j + 1
    auto stage = [&](int x) { return x % C::kStages; };
    auto phase = [&](int x) { return (uint32_t)(x / C::kStages) & 1u; };
    auto ring = [&](int x) { return sb + (uint32_t)(2 + stage(x)) * C::kTileBytes; };

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kLoadWarp) {
            // ================================ loader ================================
            if (lane == 0 && nmax > 0) {
                const int hk = h / a.G;
                auto load = [&](const CUtensorMap* m, int row, int head, uint32_t dst, int bi) {
                    mbar_expect(bar(bi), C::kTileBytes);
                    for (int x = 0; x < D / 64; ++x) tma_load3(dst + 16384u * x, m, 64 * x, head, row, bar(bi));
                };
                bool ok = true;
                int n = 0;
                for (; n < 2 * nmax; ++n) {
                    if (n >= C::kStages && !(ok = wait(B_EMPTY + stage(n), phase(n - C::kStages)))) break;
                    if (n == 0 && nb[0] > 0) load(&maps.q, q0 + r0, h, sb, B_Q);
                    load(n & 1 ? &maps.v : &maps.k, k0 + (n >> 1) * kN, hk, ring(n), B_FULL + stage(n));
                    if (n == 0 && nb[1] > 0) load(&maps.q, q0 + r0 + kM, h, sb + C::kTileBytes, B_Q + 1);
                }
                // leave no copy in flight
                for (int i = max(0, n - C::kStages); i < n; ++i) mbar_wait(bar(B_FULL + stage(i)), phase(i), kWaitNs);
                if (n > 0)
                    for (int i = 0; i < 2; ++i)
                        if (nb[i] > 0) mbar_wait(bar(B_Q + i), 0, kWaitNs);
            }
        } else if (warp == kMmaWarp) {
            // ================================ MMA issue ================================
            if (lane == 0 && nmax > 0) {
                constexpr uint32_t id_s = idesc_bf16(kM, kN, 0), id_o = idesc_bf16(kM, D, 1);
                auto s_mma = [&](int i, int j) {
                    const uint32_t q = sb + (uint32_t)i * C::kTileBytes, k = ring(2 * j);
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t o = (uint32_t)(x >> 2) * 16384u + (uint32_t)(x & 3) * 32u;
                        mma_bf16(tb + C::TS(i), sdesc(q + o, 16, 1024), sdesc(k + o, 16, 1024), id_s, x > 0);
                    }
                    mma_commit(bar(B_S + i));
                };
                bool ok = wait(B_FULL + stage(0), phase(0));
                for (int i = 0; i < 2 && ok; ++i)
                    if (nb[i] > 0) {
                        ok = wait(B_Q + i, 0);
                        fence_after();
                        if (ok) s_mma(i, 0);
                    }
                mma_commit(bar(B_EMPTY + stage(0)));
                for (int j = 0; j < nmax && ok; ++j) {
                    bool have_k = false;
                    ok = wait(B_FULL + stage(2 * j + 1), phase(2 * j + 1));
                    if (ok && j >= nf) ok = wait(B_CLEAN + stage(2 * j + 1), (uint32_t)((j - nf) / C::kCleanPeriod) & 1u);
                    for (int i = 0; i < 2 && ok; ++i) {
                        if (j < nb[i]) {
                            if (!(ok = wait(B_P + i, (uint32_t)j & 1u))) break;
                            fence_after();
                            const uint32_t v = ring(2 * j + 1);
#pragma unroll
                            for (int x = 0; x < kN / 16; ++x)
                                mma_bf16_ts(tb + C::TO(i), tb + C::TS(i) + 8 * x, sdesc(v + 2048u * x, 16384, 1024), id_o,
                                            j > 0 || x > 0);
                            mma_commit(bar(B_O + i));
                        }
                        if (j + 1 < nb[i]) {
                            if (!have_k && !(ok = wait(B_FULL + stage(2 * j + 2), phase(2 * j + 2)))) break;
                            have_k = true;
                            fence_after();
                            s_mma(i, j + 1);
                        }
                    }
                    mma_commit(bar(B_EMPTY + stage(2 * j + 1)));
                    if (j + 1 < nmax) mma_commit(bar(B_EMPTY + stage(2 * j + 2)));
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
            for (int j = 0; j < nmax && nf < nmax && ok; ++j) {
                // (every load is waited for, in order: a barrier tells only the last two phases apart)
                ok = wait(B_FULL + stage(2 * j), phase(2 * j)) && wait(B_FULL + stage(2 * j + 1), phase(2 * j + 1));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (j < nf) continue;
                uint8_t* v = sm + (size_t)(2 + stage(2 * j + 1)) * C::kTileBytes;
                const int valid = min(kN, lk - j * kN);
                bool odd = false;
                for (int x = ct; x < kN * D / 8; x += 64) {          // 16-byte chunks, in memory order
                    const int row = (x >> 3) & (kN - 1);
                    uint4* p = reinterpret_cast<uint4*>(v) + x;
                    if (row >= valid) {
                        *p = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    const uint4 y = *p;
                    uint32_t w[4] = {y.x, y.y, y.z, y.w};
                    bool hit = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const bool lo = (w[e] & 0x7f80u) == 0x7f80u, hi = (w[e] & 0x7f800000u) == 0x7f800000u;
                        hit |= lo | hi;
                        w[e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
                    }
                    if (hit) {
                        *p = make_uint4(w[0], w[1], w[2], w[3]);
                        odd = true;
                    }
                }
                if (odd) *reinterpret_cast<volatile int*>(&odd_sm) = 1;
                fence_async_smem();
                __threadfence_block();
                __syncwarp();
                if (lane == 0) mbar_arrive1(bar(B_CLEAN + stage(2 * j + 1)));
            }
        }
    } else {
        // ================================ softmax ================================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
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
                const int lim = last - j * kN;
#pragma unroll
                for (int x = 0; x < kN; ++x) s[x] = x <= lim ? s[x] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int x = 4; x < kN; ++x) mx[x & 3] = fmaxf(mx[x & 3], s[x]);
            const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            const bool need = bm > m + kRaise;
            if (j == 0) {
                m = bm;
            } else if (__any_sync(0xffffffffu, need)) {
                // O_i is quiet once the product before this block is done
                if (!(ok = __all_sync(0xffffffffu, wait(B_O + i, (uint32_t)(j - 1) & 1u)))) break;
                fence_after();
                const float f = need ? ex2(m - bm) : 1.f;
                l *= f;
#pragma unroll
                for (int x = 0; x < D; x += 32) {
                    float o[32];
                    tmem_ld32(to + x, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] *= f;
                    tmem_st32(to + x, o);
                }
                if (need) m = bm;
            }
            const float base = m == -INFINITY ? 0.f : m;
            float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < kN; x += 32) {
                uint32_t p[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    const float e0 = ex2(fmaf(s[x + 2 * y], c, -base)), e1 = ex2(fmaf(s[x + 2 * y + 1], c, -base));
                    ls[(2 * y) & 3] += e0;
                    ls[(2 * y + 1) & 3] += e1;
                    const __nv_bfloat162 bp = __floats2bfloat162_rn(e0, e1);
                    p[y] = *reinterpret_cast<const uint32_t*>(&bp);
                }
                tmem_st16(ts + x / 2, p);
            }
            l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive1(bar(B_P + i));
        }
        // ---- o = O / l ----
        if (n > 0 && ok) ok = __all_sync(0xffffffffu, wait(B_O + i, (uint32_t)(n - 1) & 1u));
        fence_after();
        const bool none = last < 0 || n == 0, live = row < lq && ok;
        const float inv = 1.f / l;
        __nv_bfloat16* O = reinterpret_cast<__nv_bfloat16*>(a.O.data) + (int64_t)(q0 + row) * a.O.row + (int64_t)h * a.O.head;
        const bool odd = *reinterpret_cast<volatile int*>(&odd_sm) != 0;
#pragma unroll
        for (int x = 0; x < D; x += 32) {
            float o[32];
            if (n > 0) {
                tmem_ld32(to + x, o);
                tmem_wait_ld();
            }
            uint32_t p[16];
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = none ? 0.f : o[y] * inv;
            if (odd && live) {
                // values that are not finite and were kept out of the products: for the keys the row sees
                const __nv_bfloat16* V = reinterpret_cast<const __nv_bfloat16*>(a.V.data) +
                                         (int64_t)(h / a.G) * a.V.head + x;
                for (int key = nf * kN; key <= last; ++key)
#pragma unroll
                    for (int y = 0; y < 32; ++y) {
                        const float v = __bfloat162float(V[(int64_t)(k0 + key) * a.V.row + y]);
                        if (!(fabsf(v) <= 3.4e38f)) o[y] += v;
                    }
            }
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                const __nv_bfloat162 bp = __floats2bfloat162_rn(o[2 * y], o[2 * y + 1]);
                p[y] = *reinterpret_cast<const uint32_t*>(&bp);
            }
            if (live) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<uint4*>(O + x + 8 * y) = make_uint4(p[4 * y], p[4 * y + 1], p[4 * y + 2], p[4 * y + 3]);
            }
        }
        if (a.lse && live)
            a.lse[(int64_t)h * a.total_q + q0 + row] = none ? -INFINITY : (m + log2f(l)) * kAttnLn2;
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (abort_sm && tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
    if (warp == kMmaWarp) tmem_dealloc<512>(tb);
}

bool make_map(CUtensorMap* m, const Rows& r, int64_t rows, int heads, int d) {
    return make_tmap_rows(m, r.data, rows, heads, d, r.row, r.head, kM);
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
    Maps maps;
    const int Hkv = a.Hq / a.G;
    const int64_t rows_k = a.total_k > 0 ? a.total_k : 1;
    if (!make_map(&maps.q, a.Q, a.total_q, a.Hq, D) || !make_map(&maps.k, a.K, rows_k, Hkv, D) ||
        !make_map(&maps.v, a.V, rows_k, Hkv, D))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_smem(attn_tc_kernel<D>, Cfg<D>::kSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((int64_t)a.total_q + (int64_t)a.n_seq * (kQ - 1)) / kQ;
    attn_tc_kernel<D><<<(unsigned)(tiles * a.Hq), kThreads, Cfg<D>::kSmem, st>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st) { return a.d == 128 ? launch<128>(a, st) : launch<64>(a, st); }

cudaError_t attn_tc_status_take(int32_t* bits, cudaStream_t st) { return take_word(g_status, bits, st); }

}  // namespace lola
