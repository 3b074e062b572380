// K8 (CUDA cores): causal softmax attention over packed prompts.
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j <= i + Lk - Lq.  One pass over
// the keys with a running maximum m and sum l per row (log2 units, s = c log2(e) q . k):
//   m' = max(m, max_j s_j),  l' = 2^{m - m'} l + sum_j 2^{s_j - m'},
//   O' = 2^{m - m'} O + sum_j 2^{s_j - m'} v_j,        o = O / l,  lse = ln 2 (m + log2 l).
// A CTA of 128 threads takes 32 queries of one head and 64 keys at a time; a thread holds a 4 x 4 tile of
// the scores and 4 rows x d / 16 columns of O.  Q and K sit in shared memory with the channel
// outermost, so that a channel's 4 + 4 operands of 16 products are two 16-byte reads.  V takes K's
// place once the scores are formed, which lets four (d = 64) or three (d = 128) CTAs share an SM: with
// 64 queries a CTA the longest one ran alone at the end (three prompts of 512-1024 tokens, 8 heads, d =
// 64: 128 us against %%).  Bound by the FMA pipe for large batches, by the longest CTA for small ones.
#include "lola_attn.cuh"

namespace lola {
namespace {

__device__ int32_t g_status;

constexpr int kTQ = 32;        // queries per tile
constexpr int kT = 64;         // keys per tile
constexpr int kNT = 128;
constexpr int kLd = kT + 4;    // row strides of the transposed tiles (16-byte aligned rows)
constexpr int kLdQ = kTQ + 4;

// R rows of one head from src on (rows from `rows` on are zero) into shared memory, transposed: channel
// c of row r at c * LD + r
template <int D, int R, int LD>
__device__ __forceinline__ void load_t(float* dst, const float* src, int64_t ld, int rows, float scale) {
    const int r = threadIdx.x % R;
#pragma unroll 4
    for (int c = threadIdx.x / R; c < D / 4; c += kNT / R) {
        const float4 v = r < rows ? *reinterpret_cast<const float4*>(src + r * ld + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        dst[(4 * c) * LD + r] = v.x * scale;
        dst[(4 * c + 1) * LD + r] = v.y * scale;
        dst[(4 * c + 2) * LD + r] = v.z * scale;
        dst[(4 * c + 3) * LD + r] = v.w * scale;
    }
}
// row-major; returns whether some value is not finite
template <int D>
__device__ __forceinline__ bool load_rows(float* dst, const float* src, int64_t ld, int rows) {
    float worst = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < kT * (D / 4); i += kNT) {
        const int r = i / (D / 4), c = i % (D / 4);
        const float4 v = r < rows ? *reinterpret_cast<const float4*>(src + r * ld + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        worst = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, worst))));   // 0 or NaN
        *reinterpret_cast<float4*>(dst + r * D + 4 * c) = v;
    }
    return worst != 0.f;
}

template <int D>
__global__ void __launch_bounds__(kNT, D == 64 ? 4 : 3) attn_prefill_kernel(const AttnArgs a) {
    using T = float;
    extern __shared__ __align__(16) float sm[];
    float* Qs = sm;                   // [D][kLdQ]
    float* Ks = Qs + D * kLdQ;        // [D][kLd], then
    float* Vs = Ks;                   // [kT][D]
    float* Ps = Ks + D * kLd;         // [key][kLdQ]
    constexpr int CW = D / 16;        // O columns per thread

    const int h = blockIdx.x % (unsigned)a.Hq;
    TilePos at;
    const bool live = find_tile<kNT, kTQ>(a, (int)(blockIdx.x / (unsigned)a.Hq), &at);
    if (at.bad) atomicOr(&g_status, (int)LOLA_ATTN_BAD_OFFSETS);
    if (!live) return;
    const int q0 = at.q0, lq = at.lq, k0 = at.k0, lk = at.lk;
    const int r0 = at.tile * kTQ, rows = min(kTQ, lq - r0), shift = lk - lq;
    const int keys = max(0, min(lk, r0 + rows + shift));      // keys some row of the tile sees

    const T* Q = reinterpret_cast<const T*>(a.Q.data) + (int64_t)(q0 + r0) * a.Q.row + (int64_t)h * a.Q.head;
    const T* K = reinterpret_cast<const T*>(a.K.data) + (int64_t)k0 * a.K.row + (int64_t)(h / a.G) * a.K.head;
    const T* V = reinterpret_cast<const T*>(a.V.data) + (int64_t)k0 * a.V.row + (int64_t)(h / a.G) * a.V.head;
    load_t<D, kTQ, kLdQ>(Qs, Q, a.Q.row, rows, a.scale_log2);

    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;   // rows 4 ty .., keys 4 tx .., columns
    float m[4], l[4], acc[4][CW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < CW; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = 0; j0 < keys; j0 += kT) {
        const int nk = min(kT, keys - j0);
        __syncthreads();
        load_t<D, kT, kLd>(Ks, K + (int64_t)j0 * a.K.row, a.K.row, nk, 1.f);
        __syncthreads();
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
        for (int c = 0; c < D; ++c) {
            const float4 q = *reinterpret_cast<const float4*>(Qs + c * kLdQ + 4 * ty);
            const float4 k = *reinterpret_cast<const float4*>(Ks + c * kLd + 4 * tx);
            const float qv[4] = {q.x, q.y, q.z, q.w}, kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = fmaf(qv[i], kv[j], s[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = r0 + 4 * ty + i + shift;         // the row's last key
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + 4 * tx + j;
                if (key > last || key >= keys) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - base);
                sum += s[i][j];
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * f + sum;
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < CW; ++c) acc[i][c] *= f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(Ps + (4 * tx + j) * kLdQ + 4 * ty) =
                make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
        __syncthreads();                                      // (K is read)
        const bool any_odd = __syncthreads_or(load_rows<D>(Vs, V + (int64_t)j0 * a.V.row, a.V.row, nk));
        if (!any_odd) {
#pragma unroll 4
            for (int j = 0; j < kT; ++j) {
                const float4 p = *reinterpret_cast<const float4*>(Ps + j * kLdQ + 4 * ty);
                const float pv[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int c4 = 0; c4 < CW / 4; ++c4) {
                    const float4 v = *reinterpret_cast<const float4*>(Vs + j * D + 64 * c4 + 4 * tx);
                    const float vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][4 * c4 + e] = fmaf(pv[i], vv[e], acc[i][4 * c4 + e]);
                }
            }
        } else {
            // a value of the tile is not finite: only the keys a row sees may touch it
            for (int j = 0; j < nk; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j0 + j <= r0 + 4 * ty + i + shift) {
                        const float p = Ps[j * kLdQ + 4 * ty + i];
#pragma unroll
                        for (int c = 0; c < CW; ++c)
                            acc[i][c] = fmaf(p, Vs[j * D + 64 * (c / 4) + 4 * tx + (c & 3)], acc[i][c]);
                    }
        }
    }
    T* O = reinterpret_cast<T*>(a.O.data) + (int64_t)(q0 + r0) * a.O.row + (int64_t)h * a.O.head;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        const bool none = r0 + r + shift < 0;                 // the row sees no key
        const float inv = 1.f / l[i];
#pragma unroll
        for (int c4 = 0; c4 < CW / 4; ++c4)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                IO<T>::st(O, r * a.O.row + 64 * c4 + 4 * tx + e, none ? 0.f : acc[i][4 * c4 + e] * inv);
        if (a.lse && tx == 0)
            a.lse[(int64_t)h * a.total_q + q0 + r0 + r] = none ? -INFINITY : (m[i] + log2f(l[i])) * kAttnLn2;
    }
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(float) * (D * kLdQ + D * kLd + kT * kLdQ);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_smem(attn_prefill_kernel<D>, (int)smem, done);
    if (e != cudaSuccess) return e;
    // at most this many tiles for any cut of total_q rows into n_seq sequences
    const int64_t tiles = ((int64_t)a.total_q + (int64_t)a.n_seq * (kTQ - 1)) / kTQ;
    attn_prefill_kernel<D><<<(unsigned)(tiles * a.Hq), kNT, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t st) {
    if (a.dtype == LOLA_F32) return a.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
    return launch_attn_tc(a, st);
}

cudaError_t attn_status_take(int32_t* bits, cudaStream_t st) { return take_word(g_status, bits, st); }

}  // namespace lola
