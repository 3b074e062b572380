// K8 (CUDA cores): causal softmax attention over packed prompts.
//
// Row i of a sequence with Lq queries and Lk keys sees the keys j <= i + Lk - Lq.  One pass over
// the keys with a running maximum m and sum l per row (log2 units, s = c log2(e) q . k):
//   m' = max(m, max_j s_j),  l' = 2^{m - m'} l + sum_j 2^{s_j - m'},
//   O' = 2^{m - m'} O + sum_j 2^{s_j - m'} v_j,        o = O / l,  lse = ln 2 (m + log2 l).
// A CTA takes 64 queries of one head and 64 keys at a time; a thread holds a 4 x 4 tile of the
// scores and 4 rows x d / 16 columns of O.  Q and K sit in shared memory with the channel
// outermost, so that a channel's 4 + 4 operands of 16 products are two 16-byte reads; FMA-bound.
#include "lola_attn.cuh"

namespace lola {
namespace {

__device__ int32_t g_status;

constexpr int kT = 64;         // queries and keys per tile
constexpr int kNT = 256;
constexpr int kLd = kT + 4;    // row stride of the transposed tiles (16-byte aligned rows)

template <typename T> struct Vec;   // 16 bytes of T as floats
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void ld(const float* p, float (&v)[4]) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void ld(const __nv_bfloat16* p, float (&v)[8]) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// 64 rows of one head from row r0 (rows from `rows` on are zero) into shared memory:
// transposed (channel c of row r at c * kLd + r)
template <typename T, int D>
__device__ __forceinline__ void load_t(float* dst, const T* src, int64_t ld, int rows, float scale) {
    constexpr int VN = Vec<T>::N, CH = D / VN;
    const int r = threadIdx.x % kT;
    for (int c = threadIdx.x / kT; c < CH; c += kNT / kT) {
        float v[VN];
        if (r < rows) {
            Vec<T>::ld(src + r * ld + c * VN, v);
        } else {
#pragma unroll
            for (int i = 0; i < VN; ++i) v[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) dst[(c * VN + i) * kLd + r] = v[i] * scale;
    }
}
// row-major; returns whether some value is not finite
template <typename T, int D>
__device__ __forceinline__ bool load_rows(float* dst, const T* src, int64_t ld, int rows) {
    constexpr int VN = Vec<T>::N, CH = D / VN;
    float worst = 0.f;
    for (int i = threadIdx.x; i < kT * CH; i += kNT) {
        const int r = i / CH, c = i % CH;
        float v[VN];
        if (r < rows) {
            Vec<T>::ld(src + r * ld + c * VN, v);
        } else {
#pragma unroll
            for (int k = 0; k < VN; ++k) v[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < VN; ++k) {
            worst = fmaf(v[k], 0.f, worst);              // 0 or NaN
            dst[r * D + c * VN + k] = v[k];
        }
    }
    return worst != 0.f;
}

template <typename T, int D>
__global__ void __launch_bounds__(kNT, 2) attn_prefill_kernel(const AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    float* Qs = sm;                   // [D][kLd]
    float* Ks = Qs + D * kLd;         // [D][kLd]
    float* Vs = Ks + D * kLd;         // [kT][D]
    float* Ps = Vs + kT * D;          // [key][kLd]
    constexpr int CW = D / 16;        // O columns per thread

    const int h = blockIdx.x % (unsigned)a.Hq;
    TilePos at;
    const bool live = find_tile<kNT, kT>(a, (int)(blockIdx.x / (unsigned)a.Hq), &at);
    if (at.bad) atomicOr(&g_status, (int)LOLA_ATTN_BAD_OFFSETS);
    if (!live) return;
    const int q0 = at.q0, lq = at.lq, k0 = at.k0, lk = at.lk;
    const int r0 = at.tile * kT, rows = min(kT, lq - r0), shift = lk - lq;
    const int keys = max(0, min(lk, r0 + rows + shift));      // keys some row of the tile sees

    const T* Q = reinterpret_cast<const T*>(a.Q.data) + (int64_t)(q0 + r0) * a.Q.row + (int64_t)h * a.Q.head;
    const T* K = reinterpret_cast<const T*>(a.K.data) + (int64_t)k0 * a.K.row + (int64_t)(h / a.G) * a.K.head;
    const T* V = reinterpret_cast<const T*>(a.V.data) + (int64_t)k0 * a.V.row + (int64_t)(h / a.G) * a.V.head;
    load_t<T, D>(Qs, Q, a.Q.row, rows, a.scale_log2);

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
        load_t<T, D>(Ks, K + (int64_t)j0 * a.K.row, a.K.row, nk, 1.f);
        const bool odd = load_rows<T, D>(Vs, V + (int64_t)j0 * a.V.row, a.V.row, nk);
        const bool any_odd = __syncthreads_or(odd);
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
        for (int c = 0; c < D; ++c) {
            const float4 q = *reinterpret_cast<const float4*>(Qs + c * kLd + 4 * ty);
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
            *reinterpret_cast<float4*>(Ps + (4 * tx + j) * kLd + 4 * ty) =
                make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
        __syncthreads();
        if (!any_odd) {
#pragma unroll 4
            for (int j = 0; j < kT; ++j) {
                const float4 p = *reinterpret_cast<const float4*>(Ps + j * kLd + 4 * ty);
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
                        const float p = Ps[j * kLd + 4 * ty + i];
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

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(float) * (2 * D * kLd + kT * D + kT * kLd);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_smem(attn_prefill_kernel<T, D>, (int)smem, done);
    if (e != cudaSuccess) return e;
    // at most this many tiles for any cut of total_q rows into n_seq sequences
    const int64_t tiles = ((int64_t)a.total_q + (int64_t)a.n_seq * (kT - 1)) / kT;
    attn_prefill_kernel<T, D><<<(unsigned)(tiles * a.Hq), kNT, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t st) {
    if (a.dtype == LOLA_F32) return a.d == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
    return launch_attn_tc(a, st);
}

cudaError_t attn_status_take(int32_t* bits, cudaStream_t st) { return take_word(g_status, bits, st); }

}  // namespace lola
