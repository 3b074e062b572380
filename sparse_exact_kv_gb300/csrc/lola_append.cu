// K9: new tokens' keys and values into the paged cache, keys (and queries) rotated on the way.
//
// A pair (a, b) of channel pair i at position p becomes (a cos x - b sin x, b cos x + a sin x),
// x = p w_i.  The angle only matters modulo one turn, so the kernel keeps W_i = frac(w_i / 2 pi)
// as a 64-bit fixed-point fraction of a turn and takes p W_i modulo 2^64: the turn's fraction to
// about 2^-56 p (from the double product w_i / 2 pi), exact in the reduction, whatever p.  Its top
// 32 bits, read as a signed fraction, go to sincospif.
//
// Bound by HBM bytes for prompts (every element read once and written once, 16-byte accesses,
// a pair's two halves in one thread) and by latency for one token per sequence (one CTA per
// token there: more CTAs, and no token waits for another's page lookup).
#include "lola_attn.cuh"

namespace lola {
namespace {

__device__ int32_t g_status;

constexpr int kNT = 128;

// the sequence that row t belongs to, one warp: the last b with cu[b] <= t, found 32 offsets at a
// time; -1 if none
__device__ __forceinline__ int warp_find_seq(const int32_t* cu, int n_seq, int t, int lane) {
    int lo = 0, hi = n_seq + 1;            // cu[lo] <= t < cu[hi] (hi may be one past the end)
    if (cu[0] > t || cu[n_seq] <= t) return -1;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool le = at < hi && cu[at] <= t;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        lo = lo + k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

template <typename T> __device__ __forceinline__ void unpack(const uint4& x, float (&v)[16 / sizeof(T)]);
template <> __device__ __forceinline__ void unpack<float>(const uint4& x, float (&v)[4]) {
    v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y); v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& x, float (&v)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <typename T> __device__ __forceinline__ uint4 pack(const float (&v)[16 / sizeof(T)]);
template <> __device__ __forceinline__ uint4 pack<float>(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <> __device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One unit of work: 2 x 16 bytes of one head of one token.
//   u < rot_units        rotated chunk pair
//   then                 copied 32-byte chunks (channels from rot on)
template <typename T, int D>
__device__ __forceinline__ void move_unit(const T* src, T* dst, int u, int rot, bool neighbours, const float2* cs) {
    constexpr int VN = 16 / sizeof(T);
    const int ru = rot / (2 * VN);
    if (u >= ru) {
        const int c = rot + (u - ru) * 2 * VN;
        const uint4 x = *reinterpret_cast<const uint4*>(src + c), y = *reinterpret_cast<const uint4*>(src + c + VN);
        *reinterpret_cast<uint4*>(dst + c) = x;
        *reinterpret_cast<uint4*>(dst + c + VN) = y;
        return;
    }
    const int c0 = neighbours ? u * 2 * VN : u * VN, c1 = neighbours ? c0 + VN : c0 + rot / 2;
    const uint4 x = *reinterpret_cast<const uint4*>(src + c0), y = *reinterpret_cast<const uint4*>(src + c1);
    float a[VN], b[VN];
    unpack<T>(x, a);
    unpack<T>(y, b);
    if (neighbours) {
        // 2 VN consecutive channels: pairs u VN .. u VN + VN - 1
#pragma unroll
        for (int i = 0; i < VN; i += 2) {
            const float2 s = cs[u * VN + i / 2], t = cs[u * VN + VN / 2 + i / 2];
            const float a0 = a[i], b0 = b[i];
            a[i] = a0 * s.x - a[i + 1] * s.y;
            a[i + 1] = a[i + 1] * s.x + a0 * s.y;
            b[i] = b0 * t.x - b[i + 1] * t.y;
            b[i + 1] = b[i + 1] * t.x + b0 * t.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const float2 s = cs[u * VN + i];
            const float a0 = a[i];
            a[i] = a0 * s.x - b[i] * s.y;
            b[i] = b[i] * s.x + a0 * s.y;
        }
    }
    *reinterpret_cast<uint4*>(dst + c0) = pack<T>(a);
    *reinterpret_cast<uint4*>(dst + c1) = pack<T>(b);
}

template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kNT) paged_append_kernel(const AppendArgs a) {
    __shared__ float2 cs[TOK][D / 2];
    __shared__ int64_t slot[TOK];      // element offset of (page, head 0, slot), -1: no slot, -2: skip the row
    __shared__ int pos_sm[TOK];
    constexpr int VN = 16 / sizeof(T), UH = D / (2 * VN);   // units per head
    const int t0 = blockIdx.x * TOK, nt = min(TOK, a.n_tokens - t0);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const PagedArgs& p = a.p;

    for (int i = warp; i < nt; i += kNT / kWarp) {
        const int t = t0 + i;
        int b = t;
        int64_t pos;
        if (a.cu_new) {
            b = warp_find_seq(a.cu_new, p.n_seq, t, lane);
            pos = b < 0 ? -1 : (int64_t)p.kv_len[b] - a.cu_new[b + 1] + t;
            if (b >= 0 && t < a.cu_new[b]) pos = -1;          // (offsets that are not sorted)
        } else {
            pos = (int64_t)p.kv_len[b] - 1;
        }
        if (lane == 0) {
            int64_t s = -2;
            if (pos >= 0) {
                const int page = pos < paged_tokens(p, p.kv_len[b]) ? paged_page(p, b, pos) : -1;
                s = page < 0 ? -1 : paged_offset(p, page, 0, pos);
                if (page < 0) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
            }
            slot[i] = s;
            pos_sm[i] = a.positions ? a.positions[t] : (int)pos;
        }
    }
    const int rot = a.inv_freq ? a.rot : 0;
    __syncthreads();
    for (int e = threadIdx.x; e < nt * (rot / 2); e += kNT) {
        const int i = e / (rot / 2), f = e % (rot / 2);
        double turns = (double)a.inv_freq[f] * 0.15915494309189535;    // w / 2 pi
        turns -= floor(turns);
        const uint64_t w = (uint64_t)(turns * 18446744073709551616.0);   // fraction of a turn, 2^-64
        const uint64_t x = w * (uint64_t)(int64_t)pos_sm[i];             // modulo one turn
        float s, c;
        sincospif((float)(int32_t)(uint32_t)(x >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        cs[i][f] = make_float2(c, s);
    }
    __syncthreads();
    const int hq = a.Q.data ? p.Hq : 0, heads = hq + 2 * p.Hkv;
    const bool nb = a.pairs == LOLA_PAIRS_NEIGHBOURS;
    for (int e = threadIdx.x; e < nt * heads * UH; e += kNT) {
        const int u = e % UH, h = (e / UH) % heads, i = e / (UH * heads);
        const int64_t t = t0 + i, s = slot[i];
        if (s == -2 || (s < 0 && h >= hq)) continue;
        if (h < hq) {
            move_unit<T, D>(reinterpret_cast<const T*>(a.Q.data) + t * a.Q.row + h * a.Q.head,
                            reinterpret_cast<T*>(a.QO.data) + t * a.QO.row + h * a.QO.head, u, rot, nb, cs[i]);
        } else if (h < hq + p.Hkv) {
            const int hk = h - hq;
            move_unit<T, D>(reinterpret_cast<const T*>(a.K.data) + t * a.K.row + hk * a.K.head,
                            reinterpret_cast<T*>(p.K) + s + (int64_t)hk * p.page * D, u, rot, nb, cs[i]);
        } else {
            const int hk = h - hq - p.Hkv;
            move_unit<T, D>(reinterpret_cast<const T*>(a.V.data) + t * a.V.row + hk * a.V.head,
                            reinterpret_cast<T*>(p.V) + s + (int64_t)hk * p.page * D, u, 0, nb, cs[i]);
        }
    }
}

template <typename T, int D>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
    paged_append_kernel<T, D, 1><<<a.n_tokens, kNT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
    return a.p.d == 128 ? launch<__nv_bfloat16, 128>(a, st) : launch<__nv_bfloat16, 64>(a, st);
}

cudaError_t append_status_take(int32_t* bits, cudaStream_t st) { return take_word(g_status, bits, st); }

}  // namespace lola
