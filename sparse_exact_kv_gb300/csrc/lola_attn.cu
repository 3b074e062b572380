// K8 (float32): causal softmax attention over packed prompts, keys and values packed too or in the pages of
// a cache.
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j <= i + Lk - Lq.  One pass over
// the keys with a running maximum m and sum l per row (log2 units, s = c log2(e) q . k):
//   m' = max(m, max_j s_j),  l' = 2^{m - m'} l + sum_j 2^{s_j - m'},
//   O' = 2^{m - m'} O + sum_j 2^{s_j - m'} v_j,        o = O / l,  lse = ln 2 (m + log2 l).
//
// Both products run on the warps' tensor instructions in tf32, every operand split as x = hi + lo with hi
// the nearest tf32 and lo = x - hi exact: a b ~ hi hi + hi lo + lo hi.  |lo| <= 2^-11 |x| has one bit more than
// tf32 holds, so what is left out of a product is lo lo (2^-22 of |a b|) and that bit twice (2^-23 each):
// 2^-21 of |a b| at most, about a float32 product's rounding in the mean.  The instruction cuts its sums off
// instead of rounding them: a running output kept in its accumulators loses part of a last place every step,
// always towards zero (16000 keys: 1e-5 of the output, float32 sums 3e-7).  So it only adds 16 keys of the
// output, and half of the channels of a score, and those sums are added in float32, rounded (2e-7; 65 -> 67 us for
// three prompts of 512-1024 tokens, 8/2 heads, d = 64, and 111 -> 123 us at d = 128).  CUDA cores need two
// shared-memory reads for 16 products here and were bound by those (31 TFLOP/s at d = 128, half of the FMA rate
// at best); the tensor form reads an operand once for 16 rows.
//
// A CTA of four warps takes 32 queries of one head and 32 keys at a time, two tiles of K and V in flight
// (cp.async): 16 queries and 16 keys of every tile a warp, the two halves of a query's keys joined at the
// end (a warp that sees all keys of 16 queries is alone with the longest prompts: 78 us against 62 for
// three prompts of 512-1024 tokens, 8 heads, d = 64).  Bound by the instruction's rate, about 256 multiply-adds
// a cycle and SM, and the splits beside it: 49 TFLOP/s of attention, 146 of products (4000 tokens, 16 heads, d = 64).
// Rows of 4 floats more than d keep every fragment read free of bank conflicts: K's (key = lane / 4, channel =
// lane % 4) and V's (key = 2 (lane % 4), channel = lane / 4), where keys 2 t and 2 t + 1 stand in for the
// instruction's rows t and t + 4, so that the scores' accumulators are the weights' operand as they stand.
#include "lola_attn.cuh"
#include "lola_tc.cuh"

namespace lola {
namespace {

__device__ int32_t g_status;

constexpr int kTQ = 32;        // queries per CTA
constexpr int kT = 32;         // keys per tile
constexpr int kTW = kT / 2;    // ... of a warp
constexpr int kNT = 128;

__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
    // (an infinity or NaN leaves a NaN in lo: the callers look for them)
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
// ... of a value: hi stops at the largest finite tf32, so that the finite values above it (from 0x7f7ff000 on, which
// round to infinity) keep finite parts.  Scores need no such stop: those that come out NaN are formed again.
__device__ __forceinline__ void split_value(float x, uint32_t& hi, uint32_t& lo) {
    const float r = __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u);
    float h;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(h) : "f"(r), "f"(__uint_as_float(0x7f7fe000u)));   // the smaller magnitude, r's sign
    hi = __float_as_uint(h);
    lo = __float_as_uint(x - h);
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// PG: keys and values in the pages of a cache
template <int D, bool PG>
__global__ void __launch_bounds__(kNT, D == 64 ? 3 : 2) attn_f32_kernel(const AttnArgs a) {
    constexpr int LD = D + 4, TILE = kT * LD;
    extern __shared__ __align__(16) float sm[];       // [2][K, V][kT][LD]
    wait_for_last_kernel();
    const int h = blockIdx.x % (unsigned)a.Hq, hk = h / a.G;
    TilePos at;
    const bool live = find_tile<kNT, kTQ, PG>(a, (int)(blockIdx.x / (unsigned)a.Hq), &at);
    if (at.bits) atomicOr(&g_status, at.bits);
    if (!live) return;
    const int q0 = at.q0, lq = at.lq, k0 = at.k0, lk = at.lk, shift = lk - lq;
    const int r0 = at.tile * kTQ, rows = min(kTQ, lq - r0);
    const int keys = max(0, min(lk, r0 + rows + shift));      // keys some row of the tile sees
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane >> 2, t = lane & 3;
    const int row0 = r0 + 16 * (warp & 1) + g;                // this thread's rows: row0, row0 + 8
    const int kw = (warp >> 1) * kTW;                         // this warp's keys of a tile
    const int last[2] = {min(row0 + shift, lk - 1), min(row0 + 8 + shift, lk - 1)};   // their last keys

    const float* Q = reinterpret_cast<const float*>(a.Q.data) + (int64_t)q0 * a.Q.row + (int64_t)h * a.Q.head;
    const float *K, *V;
    if constexpr (PG) {
        K = reinterpret_cast<const float*>(a.p.K);
        V = reinterpret_cast<const float*>(a.p.V);
    } else {
        K = reinterpret_cast<const float*>(a.K.data) + (int64_t)k0 * a.K.row + (int64_t)hk * a.K.head;
        V = reinterpret_cast<const float*>(a.V.data) + (int64_t)k0 * a.V.row + (int64_t)hk * a.V.head;
    }
    // the pages of a tile's halves, looked up one tile ahead; -1: none, or not in the cache
    int pages[2] = {-1, -1};
    auto look_up = [&](int j) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int pos = j * kT + x * 16;
            pages[x] = pos < keys ? paged_page(a.p, at.b, pos) : -1;
            if (pos < keys && pages[x] < 0) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
        }
    };
    // tile j into its half of shared memory; rows behind the keys are zeros, and those without a page
    auto load = [&](int j) {
        float* dst = sm + (j & 1) * 2 * TILE;
#pragma unroll
        for (int x = 0; x < kT * D / 4 / kNT; ++x) {
            const int e = threadIdx.x + x * kNT, r = e / (D / 4), c = e % (D / 4) * 4, key = j * kT + r;
            if constexpr (PG) {
                const int page = r < 16 ? pages[0] : pages[1];
                const uint32_t n = key < keys && page >= 0 ? 16u : 0u;
                const int64_t src = n ? paged_offset(a.p, page, hk, key) + c : 0;
                tc::cp_async16_z(tc::smem_u32(dst + r * LD + c), K + src, n);
                tc::cp_async16_z(tc::smem_u32(dst + TILE + r * LD + c), V + src, n);
            } else {
                const uint32_t n = key < keys ? 16u : 0u;
                const int64_t src = n ? key : 0;
                tc::cp_async16_z(tc::smem_u32(dst + r * LD + c), K + src * a.K.row + c, n);
                tc::cp_async16_z(tc::smem_u32(dst + TILE + r * LD + c), V + src * a.V.row + c, n);
            }
        }
        if constexpr (PG) look_up(j + 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int tiles = (keys + kT - 1) / kT;
    if constexpr (PG) look_up(0);
    if (tiles > 0) load(0);
    float q[D / 8][4];                                        // this warp's rows as the A operand, scaled
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = row0 + 8 * (e & 1);
            q[x][e] = r < lq ? Q[(int64_t)r * a.Q.row + 8 * x + t + 4 * (e >> 1)] * a.scale_log2 : 0.f;
        }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][e] = 0.f;
    for (int j = 0; j < tiles; ++j) {
        if (j + 1 < tiles) load(j + 1);
        else asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const float* Ks = sm + (j & 1) * 2 * TILE;
        float* Vs = sm + (j & 1) * 2 * TILE + TILE;
        // values that are not finite (x 0 is then not 0) would reach rows that do not see them
        float worst = 0.f;
#pragma unroll
        for (int x = 0; x < kT * D / 4 / kNT; ++x) {
            const int e = threadIdx.x + x * kNT;
            const float4 v = *reinterpret_cast<const float4*>(Vs + e / (D / 4) * LD + e % (D / 4) * 4);
            worst = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, worst))));
        }
        // ---- S: 16 rows x 16 keys, the channels in two halves ----
        float s[kTW / 8][4] = {}, s1[kTW / 8][4] = {}, sl[kTW / 8][4] = {};
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split(q[x][e], ah[e], al[e]);
#pragma unroll
            for (int n = 0; n < kTW / 8; ++n) {
                const float* kp = Ks + (kw + 8 * n + g) * LD + 8 * x + t;
                uint32_t h0, l0, h1, l1;
                split(kp[0], h0, l0);
                split(kp[4], h1, l1);
                mma_tf32(sl[n], ah, l0, l1);
                mma_tf32(sl[n], al, h0, h1);
                mma_tf32(x < D / 16 ? s[n] : s1[n], ah, h0, h1);
            }
        }
        bool nan = false;
#pragma unroll
        for (int n = 0; n < kTW / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[n][e] += s1[n][e] + sl[n][e];
                nan |= s[n][e] != s[n][e];
            }
        if (__any_sync(0xffffffffu, nan)) {
            // a query or key is not finite, or its upper part is not: these scores, and no others (a row's bits are
            // not to depend on keys that it does not see), once more, term by term
#pragma unroll
            for (int n = 0; n < kTW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = row0 + 8 * (e >> 1);
                    const float* kp = Ks + (kw + 8 * n + 2 * t + (e & 1)) * LD;
                    if (s[n][e] == s[n][e]) continue;
                    float x = 0.f;
                    if (r < lq)
#pragma unroll 1
                        for (int c = 0; c < D; ++c) x = fmaf(Q[(int64_t)r * a.Q.row + c] * a.scale_log2, kp[c], x);
                    s[n][e] = x;
                }
        }
        // ---- masks, running maximum, weights ----
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float mx = -INFINITY;
#pragma unroll
            for (int n = 0; n < kTW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (j * kT + kw + 8 * n + 2 * t + e > last[r]) s[n][2 * r + e] = -INFINITY;
                    mx = fmaxf(mx, s[n][2 * r + e]);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[r] - base);
            m[r] = mn;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < kTW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s[n][2 * r + e] = exp2f(s[n][2 * r + e] - base);
                    sum += s[n][2 * r + e];
                }
            l[r] = l[r] * f + sum;                            // (this thread's keys; joined at the end)
            if (__any_sync(0xffffffffu, f != 1.f))
#pragma unroll
                for (int x = 0; x < D / 8; ++x) {
                    o[x][2 * r] *= f;
                    o[x][2 * r + 1] *= f;
                }
        }
        const bool odd = __syncthreads_or(worst != 0.f);
        if (odd) {
            for (int e = threadIdx.x; e < kT * D; e += kNT) {
                float* v = Vs + e / D * LD + e % D;
                if (!(fabsf(*v) <= 3.402823466e38f)) *v = 0.f;
            }
            __syncthreads();
        }
        // ---- O += P V: keys 2 t and 2 t + 1 of eight as the instruction's t and t + 4 ----
        // (four channel groups side by side, so that their products do not wait for each other: one at a time 71 us)
        uint32_t ph[kTW / 8][4], pl[kTW / 8][4];
#pragma unroll
        for (int n = 0; n < kTW / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) split(s[n][2 * (e & 1) + (e >> 1)], ph[n][e], pl[n][e]);
#pragma unroll
        for (int x = 0; x < D / 8; x += 4) {
            float c[4][4] = {};
#pragma unroll
            for (int n = 0; n < kTW / 8; ++n) {
                uint32_t h0[4], l0[4], h1[4], l1[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float* vp = Vs + (kw + 8 * n + 2 * t) * LD + g + 8 * (x + y);
                    split_value(vp[0], h0[y], l0[y]);
                    split_value(vp[LD], h1[y], l1[y]);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) mma_tf32(c[y], ph[n], l0[y], l1[y]);
#pragma unroll
                for (int y = 0; y < 4; ++y) mma_tf32(c[y], pl[n], h0[y], h1[y]);
#pragma unroll
                for (int y = 0; y < 4; ++y) mma_tf32(c[y], ph[n], h0[y], h1[y]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x + y][e] += c[y][e];
        }
        if (odd) {
            // what was zeroed, for the keys a row sees
#pragma unroll 1
            for (int k = kw; k < kw + kTW && j * kT + k < keys; ++k) {
                const float* row;
                if constexpr (PG) {
                    const int page = paged_page(a.p, at.b, j * kT + k);
                    if (page < 0) continue;
                    row = V + paged_offset(a.p, page, hk, j * kT + k);
                } else {
                    row = V + (int64_t)(j * kT + k) * a.V.row;
                }
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = row[8 * x + 2 * t + (e & 1)];
                        if (!(fabsf(v) <= 3.402823466e38f) && j * kT + k <= last[e >> 1]) o[x][e] += v;
                    }
            }
        }
        __syncthreads();                                      // (the tile is read)
    }
    // ---- the two halves of the keys: warps 2, 3 hand theirs to warps 0, 1 ----
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    float* half = sm + (warp & 1) * 16 * (D + 2);             // o, m, l of 16 rows (lane by lane, not by row)
    if (warp >= 2) {
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) half[(4 * x + e) * 32 + lane] = o[x][e];
        if (t == 0)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                half[16 * D + 8 * r + g] = m[r];
                half[16 * D + 16 + 8 * r + g] = l[r];
            }
    }
    __syncthreads();
    if (warp >= 2) return;
    float* O = reinterpret_cast<float*>(a.O.data) + (int64_t)q0 * a.O.row + (int64_t)h * a.O.head;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = row0 + 8 * r;
        const float m1 = half[16 * D + 8 * r + g], l1 = half[16 * D + 16 + 8 * r + g];
        const float mn = fmaxf(m[r], m1), base = mn == -INFINITY ? 0.f : mn;
        const float f0 = exp2f(m[r] - base), f1 = exp2f(m1 - base), ls = l[r] * f0 + l1 * f1;
        if (row >= lq) continue;
        const bool none = last[r] < 0;                        // the row sees no key
        const float inv = 1.f / ls;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                y[e] = none ? 0.f : (o[x][2 * r + e] * f0 + half[(4 * x + 2 * r + e) * 32 + lane] * f1) * inv;
            *reinterpret_cast<float2*>(O + (int64_t)row * a.O.row + 8 * x + 2 * t) = make_float2(y[0], y[1]);
        }
        if (a.lse && t == 0)
            a.lse[(int64_t)h * a.total_q + q0 + row] = none ? -INFINITY : (mn + log2f(ls)) * kAttnLn2;
    }
}

template <int D, bool PG>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(float) * 4 * kT * (D + 4);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_smem(attn_f32_kernel<D, PG>, (int)smem, done);
    if (e != cudaSuccess) return e;
    // at most this many tiles for any cut of total_q rows into n_seq sequences
    const int64_t tiles = ((int64_t)a.total_q + (int64_t)a.n_seq * (kTQ - 1)) / kTQ;
    return launch_behind(attn_f32_kernel<D, PG>, (unsigned)(tiles * a.Hq), kNT, smem, st, a);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t st) {
    if (a.dtype == LOLA_BF16) return launch_attn_tc(a, st);
    if (a.p.table) return a.d == 128 ? launch<128, true>(a, st) : launch<64, true>(a, st);
    return a.d == 128 ? launch<128, false>(a, st) : launch<64, false>(a, st);
}

cudaError_t attn_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
