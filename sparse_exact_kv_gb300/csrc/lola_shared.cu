// K13: single-token attention of sequences that begin with common tokens (lola_shared_decode).
//
// One kernel over the prefixes (lola_prefix.cu; in float32 K10 and K11 over 16 rows at a time) and one over the
// sequences' own tokens (K10, K11) leave the parts of every row's softmax that their pieces of the work have; the
// kernel here joins them:
//   m = max_k m_k,  l = sum_k 2^{m_k - m} l_k,  o = sum_k 2^{m_k - m} z_k / l,
// the prefix' parts first, in the order of the pieces: the same inputs give the same bits.
// Bound by its chain of accesses (which parts, the parts): two rows a CTA, their parts dealt out to eight warps,
// which have three of them in flight each (64 sequences behind 16001 tokens, 32 heads, 19 prefix parts a row: 10 us).
// (When the kernel over the own tokens read the prefix' parts itself, row after row, 64 sequences behind 16001 tokens took
// it 92 us, 8 heads, d = 128.)
// Three kernels take 20 us whatever there is to do; few tokens altogether go to K10's and K11's kernels in a form whose
// sequences' tiles are those of the prefix, then their own (PRE).
#include <algorithm>

#include "lola_paged.cuh"

namespace lola {
namespace {

struct JoinArgs {
    PagedArgs p, prefix;
    const int32_t* cu;
    Parts a, b;              // of the prefixes, of the own tokens
    Rows O;
    float* lse;
};

// The prefix of sequence b (one warp), if it has one with tokens, or -1.  A prefix has sequence b if its own two offsets say
// so, whatever the others are, as for the kernels before.
__device__ __forceinline__ int prefix_of(const JoinArgs& a, int b, int lane) {
    const int n = a.prefix.n_seq;
    auto holds = [&](int begin, int end) { return begin >= 0 && begin <= b && b < end && end <= a.p.n_seq; };
    int g = 0;
    if (a.cu && n < kWarp) {
        // (few prefixes: all offsets and lengths at once)
        const int c = lane <= n ? a.cu[lane] : 0x7fffffff, len = lane < n ? a.prefix.kv_len[lane] : 0;
        const int end = __shfl_down_sync(0xffffffffu, c, 1);
        g = 31 - __clz(__ballot_sync(0xffffffffu, lane < n && holds(c, end)));
        const int tokens = __shfl_sync(0xffffffffu, len, max(g, 0));
        return g >= 0 && paged_tokens(a.prefix, tokens) > 0 ? g : -1;
    }
    if (a.cu) {
        g = warp_find_seq(a.cu, n, b, lane);
        if (g < 0 || g >= n || !holds(a.cu[g], a.cu[g + 1])) {
            // (none, or offsets that do not increase: all of them)
            int own = -1;
#pragma unroll 4
            for (int x = lane; x < n; x += kWarp)
                if (holds(a.cu[x], a.cu[x + 1])) own = x;
            g = __reduce_max_sync(0xffffffffu, own);
            if (g < 0) return -1;
        }
    }
    return paged_tokens(a.prefix, a.prefix.kv_len[g]) > 0 ? g : -1;
}
// A row's parts: none where the kernel before, whose waits gave up, has left anything else.
__device__ __forceinline__ int part_count(const Parts& q, const int4& at) {
    if (at.x == 1) return 1;
    const bool fine = at.x >= 2 && at.x <= kPieces && at.y >= 0 && at.w >= 1 && at.w <= kPieces && at.y / 2 + (at.x - 1) * at.w < kPieces &&
                      at.z >= 0 && at.z < q.rows;
    return fine ? at.x : 0;
}
// Part k of row i: where its output's first columns, m and l are, and the floats from four columns to the next.
struct Part {
    const float *z, *m, *l;
    int step;
};
__device__ __forceinline__ Part part_of(const Parts& q, const int4& at, int64_t i, int k, int d) {
    if (at.x == 1) return Part{q.whole + i * d, &q.ml[i].x, &q.ml[i].y, 4};
    const float* rec = q.rec + (int64_t)(k == 0 ? at.y : (at.y / 2 + k * at.w) * 2) * part_record(q.rows, d);
    return Part{rec + at.z * q.row_step, rec + q.rows * d + at.z, rec + q.rows * d + q.rows + at.z, q.chunk_step};
}
// One more part of a row's softmax.
template <int N> __device__ __forceinline__ void add_part(float m, float l, const float4 (&z)[N], float4 (&y)[N], float& M, float& L) {
    const float top = fmaxf(M, m), base = top == -INFINITY ? 0.f : top, f = ex2(M - base), f1 = ex2(m - base);
    L = fmaf(f, L, f1 * l);
#pragma unroll
    for (int x = 0; x < N; ++x)
        y[x] = make_float4(fmaf(f, y[x].x, f1 * z[x].x), fmaf(f, y[x].y, f1 * z[x].y), fmaf(f, y[x].z, f1 * z[x].z), fmaf(f, y[x].w, f1 * z[x].w));
    M = top;
}

// Two rows a warp, in the lanes by turns (neighbouring rows' 16 bytes of a record share a sector).
template <typename T, int D>
__global__ void __launch_bounds__(256, 4) shared_join_kernel(const JoinArgs a) {
    constexpr int N = D / 64, kWarps = 8, kBatch = 3;                    // float4 of a lane; warps; parts in flight
    __shared__ float4 y_sm[kWarps][N][kWarp];
    __shared__ float2 ml_sm[kWarps][2];
    const int w = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, own = lane >> 1;
    // (2^28 rows at most)
    const int rows = a.p.n_seq * a.p.Hq, i0 = (int)blockIdx.x * 2, i = i0 + (lane & 1);
    const int b0 = i0 / a.p.Hq, b1 = i0 + 1 < rows && i0 + 1 == (b0 + 1) * a.p.Hq ? b0 + 1 : b0, b = lane & 1 ? b1 : b0;
    wait_for_last_kernel();
    int4 at_a = make_int4(0, 0, 0, 0), at_b = at_a;
    if (i < rows) {
        at_a = __ldcg(a.a.desc + i);
        at_b = __ldcg(a.b.desc + i);
    }
    const bool has_own = paged_tokens(a.p, a.p.kv_len[b]) > 0;
    int g = prefix_of(a, b0, lane);
    if (b1 != b0) {
        const int g1 = prefix_of(a, b1, lane);
        if (lane & 1) g = g1;
    }
    const int na = i < rows && g >= 0 ? part_count(a.a, at_a) : 0, n = na + (i < rows && has_own ? part_count(a.b, at_b) : 0);
    const int most = max(n, __shfl_xor_sync(0xffffffffu, n, 1));
    float M = -INFINITY, L = 0.f;
    float4 y[N];
#pragma unroll
    for (int x = 0; x < N; ++x) y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = w; k0 < most; k0 += kWarps * kBatch) {
        float m[kBatch], l[kBatch];
        float4 z[kBatch][N];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int k = k0 + kWarps * e;
            m[e] = -INFINITY;
            if (k < n) {
                const Part q = k < na ? part_of(a.a, at_a, i, k, D) : part_of(a.b, at_b, i, k - na, D);
                m[e] = __ldcg(q.m);
                l[e] = __ldcg(q.l);
#pragma unroll
                for (int x = 0; x < N; ++x) z[e][x] = __ldcg(reinterpret_cast<const float4*>(q.z + (own + 16 * x) * q.step));
            }
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
            if (k0 + kWarps * e < n) add_part<N>(m[e], l[e], z[e], y, M, L);
    }
#pragma unroll
    for (int x = 0; x < N; ++x) y_sm[w][x][lane] = y[x];
    if (own == 0) ml_sm[w][lane & 1] = make_float2(M, L);
    __syncthreads();
    if (w > 0 || i >= rows) return;
#pragma unroll
    for (int e = 1; e < kWarps; ++e) {
        float4 z[N];
#pragma unroll
        for (int x = 0; x < N; ++x) z[x] = y_sm[e][x][lane];
        const float2 ml = ml_sm[e][lane & 1];
        add_part<N>(ml.x, ml.y, z, y, M, L);
    }
    // (no token seen: o = 0; scores that are all minus infinity: 0 / 0)
    const float inv = L == 0.f ? (sees_token(a.p, b) || (g >= 0 && sees_token(a.prefix, g)) ? NAN : 0.f) : 1.f / L;
    const int h = i - b * a.p.Hq;
    T* o = reinterpret_cast<T*>(a.O.data) + (int64_t)b * a.O.row + (int64_t)h * a.O.head;
#pragma unroll
    for (int x = 0; x < N; ++x) {
        const float v[4] = {y[x].x * inv, y[x].y * inv, y[x].z * inv, y[x].w * inv};
        store4(o + 4 * (own + 16 * x), v);
    }
    if (a.lse && own == 0) a.lse[i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kAttnLn2;
}

// ---- the workspace: the two kernels' parts ----
// Lays one kernel's out from `base` on; the bytes.
int64_t carve(Parts* q, char* base, int64_t n, int d, bool tc) {
    const int rows = tc ? kPrefixRows : kRows;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        char* x = base ? base + at : nullptr;
        at += (bytes + 15) / 16 * 16;
        return x;
    };
    q->desc = reinterpret_cast<int4*>(take(n * sizeof(int4)));
    q->ml = reinterpret_cast<float2*>(take(n * sizeof(float2)));
    q->whole = reinterpret_cast<float*>(take(n * d * sizeof(float)));
    q->rec = reinterpret_cast<float*>(take(kPieces * 2 * part_record(rows, d) * sizeof(float)));
    q->rows = rows;
    q->row_step = tc ? 4 : d;
    q->chunk_step = tc ? 4 * kPrefixRows : 4;
    return at;
}
int64_t carve(Parts* prefix, Parts* own, char* base, int n_seq, int Hq, int d, int dtype) {
    const int64_t n = (int64_t)n_seq * Hq, at = carve(prefix, base, n, d, dtype == LOLA_BF16);
    return at + carve(own, base ? base + at : nullptr, n, d, false);
}

DecodeArgs parts_args(const SharedArgs& a, bool own) {
    DecodeArgs d;
    Parts x[2];
    carve(&x[0], &x[1], a.workspace, a.p.n_seq, a.p.Hq, a.p.d, a.p.dtype);
    d.p = own ? a.p : a.prefix;
    d.pre = PagedArgs{};
    d.sh = Sharing{own ? nullptr : a.cu, a.p.n_seq, own};
    d.parts = x[own];
    d.Q = a.Q;
    d.O = a.O;
    d.lse = nullptr;
    d.part = nullptr;
    d.tag = 0;
    d.give_up = a.give_up;
    d.scale_log2 = a.scale_log2;
    return d;
}

}  // namespace

int64_t shared_workspace(int n_seq, int Hq, int d, int dtype) {
    Parts x, y;
    return std::max(carve(&x, &y, nullptr, n_seq, Hq, d, dtype), paged_decode_workspace(d));
}

cudaError_t launch_shared_prefix(const SharedArgs& a, cudaStream_t st) {
    const DecodeArgs d = parts_args(a, false);
    if (a.p.dtype == LOLA_BF16) return launch_prefix_tc(d, st);
    return a.p.Ks ? launch_quant_parts(d, st) : launch_f32_parts(d, st);
}

cudaError_t launch_shared_own(const SharedArgs& a, cudaStream_t st) {
    const DecodeArgs d = parts_args(a, true);
    const cudaError_t e = a.p.Ks ? launch_quant_parts(d, st) : a.p.dtype == LOLA_BF16 ? launch_bf16_parts(d, st) : launch_f32_parts(d, st);
    if (e != cudaSuccess) return e;
    JoinArgs j;
    j.p = a.p;
    j.prefix = a.prefix;
    j.cu = a.cu;
    carve(&j.a, &j.b, a.workspace, a.p.n_seq, a.p.Hq, a.p.d, a.p.dtype);
    j.O = a.O;
    j.lse = a.lse;
    const unsigned grid = (unsigned)(((int64_t)a.p.n_seq * a.p.Hq + 1) / 2);
    if (a.p.dtype == LOLA_F32)
        return a.p.d == 128 ? launch_behind(shared_join_kernel<float, 128>, grid, 256, 0, st, j)
                            : launch_behind(shared_join_kernel<float, 64>, grid, 256, 0, st, j);
    return a.p.d == 128 ? launch_behind(shared_join_kernel<__nv_bfloat16, 128>, grid, 256, 0, st, j)
                        : launch_behind(shared_join_kernel<__nv_bfloat16, 64>, grid, 256, 0, st, j);
}

}  // namespace lola
