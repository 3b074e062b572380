// K9: new tokens' keys and values into the paged cache, keys (and queries) rotated on the way.
//
// A pair (a, b) of channel pair i at position p becomes (a cos x - b sin x, b cos x + a sin x),
// x = p w_i.  The angle only matters modulo one turn, so the kernel keeps W_i = frac(w_i / 2 pi)
// as a 64-bit fixed-point fraction of a turn and takes p W_i modulo 2^64: the turn's fraction to
// about 2^-56 p (from the double product w_i / 2 pi), exact in the reduction, whatever p.  Its top 32 bits
// are taken to the nearest quarter turn as an integer, and only the rest, an eighth of a turn at most, becomes a
// float32 number and goes to sincospif: it is then good to 2^-27 half turns (a whole turn in float32: 2^-25, cosines
// 1.2e-7 off where their own rounding is 3e-8).
//
// Bound by HBM bytes for prompts (every element read once and written once, 16-byte accesses,
// a pair's two halves in one thread, three such units in flight a thread; 18 k tokens of 32/8 heads:
// 74.5 us, 5.9 TB/s, 88 % of the measured copy rate) and by latency for one token per sequence (3.4 us
// for 64).  The cosines of a token are formed once and read side by side by the lanes (eight reads of
// 8 bytes a unit, four ways into the same banks, took 24 us of 98 more).
#include "lola_attn.cuh"

namespace lola {
namespace {

__device__ int32_t g_status;

constexpr int kFew = 760;   // tokens up to which a CTA takes one (five CTAs per SM)

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

// One unit of work: 2 x 16 bytes of one head of one token -- a chunk of a rotated pair's first channels and
// the one of its second channels, or (from channel `rot` on) 32 bytes to copy.
template <typename T> struct Unit {
    const float4* cs;    // the unit's first two (cos, sin) pairs; null: copied
    T* dst;              // null: nothing to do
    int c0, c1;          // channels of the two chunks
    uint4 x, y;
};
// cs: float4 (i, u) at i * units + u holds pairs 2 i and 2 i + 1 of unit u, so that the lanes of a warp,
// whose units follow each other, read side by side
template <typename T>
__device__ __forceinline__ void load_unit(Unit<T>& n, const T* src, T* dst, int u, int rot, bool neighbours, const float4* cs) {
    constexpr int VN = 16 / sizeof(T);
    const int ru = rot / (2 * VN);
    const bool turn = u < ru;
    n.c0 = turn && !neighbours ? u * VN : u * 2 * VN;      // (copied: rot + 2 VN (u - ru) = 2 VN u)
    n.c1 = turn && !neighbours ? n.c0 + rot / 2 : n.c0 + VN;
    n.cs = turn ? cs + u : nullptr;
    n.dst = dst;
    n.x = *reinterpret_cast<const uint4*>(src + n.c0);
    n.y = *reinterpret_cast<const uint4*>(src + n.c1);
}
template <typename T>
__device__ __forceinline__ void finish_unit(Unit<T>& n, bool neighbours, int step) {
    constexpr int VN = 16 / sizeof(T);
    if (n.cs) {
        float a[VN], b[VN];
        unpack<T>(n.x, a);
        unpack<T>(n.y, b);
#pragma unroll
        for (int i = 0; i < VN / 2; ++i) {
            const float4 c = n.cs[i * step];
            // pairs 2 i and 2 i + 1: neighbours in the 2 VN channels, or element 2 i (+ 1) of either chunk
            auto turn = [](float& x, float& y, float co, float si) {
                const float x0 = x;
                x = x0 * co - y * si;
                y = y * co + x0 * si;
            };
            if (neighbours) {
                float(&z)[VN] = 4 * i < VN ? a : b;
                turn(z[4 * i % VN], z[4 * i % VN + 1], c.x, c.y);
                turn(z[4 * i % VN + 2], z[4 * i % VN + 3], c.z, c.w);
            } else {
                turn(a[2 * i], b[2 * i], c.x, c.y);
                turn(a[2 * i + 1], b[2 * i + 1], c.z, c.w);
            }
        }
        n.x = pack<T>(a);
        n.y = pack<T>(b);
    }
    *reinterpret_cast<uint4*>(n.dst + n.c0) = n.x;
    *reinterpret_cast<uint4*>(n.dst + n.c1) = n.y;
}

// TOK tokens a CTA of NT threads; a thread has IN units in flight.
template <typename T, int D, int TOK, int NT, int IN>
__global__ void __launch_bounds__(NT) paged_append_kernel(const AppendArgs a) {
    __shared__ __align__(16) float4 cs[TOK][D / 4];
    __shared__ uint64_t turn_sm[D / 2];
    __shared__ int64_t slot[TOK];      // element offset of (page, head 0, slot), -1: no slot, -2: skip the row
    __shared__ int pos_sm[TOK];
    constexpr int VN = 16 / sizeof(T), UH = D / (2 * VN);   // units per head
    const int t0 = blockIdx.x * TOK, nt = min(TOK, a.n_tokens - t0);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const PagedArgs& p = a.p;

    wait_for_last_kernel();
    for (int i = warp; i < nt; i += NT / kWarp) {
        const int t = t0 + i;
        int b = t;
        int64_t pos;
        if (a.cu_new) {
            b = warp_find_seq(a.cu_new, p.n_seq, t, lane);
            pos = b < 0 ? -1 : (int64_t)p.kv_len[b] - a.cu_new[b + 1] + t;
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
    // the turn of one position, by the last warps (the first ones look the tokens up)
    for (int f = NT - 1 - (int)threadIdx.x; f < rot / 2; f += NT) {
        double turns = (double)a.inv_freq[f] * 0.15915494309189535;    // w / 2 pi
        turns -= floor(turns);
        turn_sm[f] = (uint64_t)(turns * 18446744073709551616.0);         // fraction of a turn, 2^-64
    }
    __syncthreads();
    const int ru = rot / (2 * VN);
    for (int e = threadIdx.x; e < nt * (rot / 2); e += NT) {
        const int i = TOK == 1 ? 0 : e / (rot / 2), f = e - i * (rot / 2);
        const uint64_t x = turn_sm[f] * (uint64_t)(int64_t)pos_sm[i];    // modulo one turn
        float s, c;
        // the nearest quarter turn and the rest, at most an eighth of a turn either way
        const uint32_t z = (uint32_t)(x >> 32), quarter = (z + 0x20000000u) >> 30;
        sincospif((float)(int32_t)(z - (quarter << 30)) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        if (quarter & 1) {
            const float y = c;
            c = -s;
            s = y;
        }
        if (quarter & 2) c = -c, s = -s;
        reinterpret_cast<float2*>(cs[i])[((f % VN / 2) * ru + f / VN) * 2 + (f & 1)] = make_float2(c, s);
    }
    __syncthreads();
    const int hq = a.Q.data ? p.Hq : 0, heads = hq + 2 * p.Hkv, units = nt * heads * UH;
    const bool nb = a.pairs == LOLA_PAIRS_NEIGHBOURS;
    for (int e0 = threadIdx.x; e0 < units; e0 += NT * IN) {
        Unit<T> n[IN];
#pragma unroll
        for (int x = 0; x < IN; ++x) {
            const int e = e0 + x * NT;
            n[x].dst = nullptr;
            if (e >= units) continue;
            const int u = e % UH, th = e / UH;
            int i = 0;                           // th / heads
#pragma unroll
            for (int z = 1; z < TOK; ++z) i += th >= z * heads;
            const int h = th - i * heads;
            const int64_t t = t0 + i, s = slot[i];
            if (s == -2 || (s < 0 && h >= hq)) continue;
            if (h < hq) {
                load_unit<T>(n[x], reinterpret_cast<const T*>(a.Q.data) + t * a.Q.row + h * a.Q.head,
                             reinterpret_cast<T*>(a.QO.data) + t * a.QO.row + h * a.QO.head, u, rot, nb, cs[i]);
            } else {
                const bool v = h >= hq + p.Hkv;
                const int hk = h - hq - (v ? p.Hkv : 0);
                const Rows& r = v ? a.V : a.K;
                load_unit<T>(n[x], reinterpret_cast<const T*>(r.data) + t * r.row + hk * r.head,
                             reinterpret_cast<T*>(v ? p.V : p.K) + s + (int64_t)hk * p.page * D, u, v ? 0 : rot, nb, cs[i]);
            }
        }
#pragma unroll
        for (int x = 0; x < IN; ++x)
            if (n[x].dst) finish_unit<T>(n[x], nb, ru);
    }
}

// Few tokens: one a CTA, so that none waits for another's page lookup; many: four, whose rows of a head
// lie side by side in the page (512 tokens, 32/8 heads: 4.5 us one a CTA, 5.5 us four; 1024: 7.4 and 6.6).
template <typename T, int D>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
    if (a.n_tokens <= kFew) return launch_behind(paged_append_kernel<T, D, 1, 128, 3>, (unsigned)a.n_tokens, 128, 0, st, a);
    return launch_behind(paged_append_kernel<T, D, 4, 256, 3>, (unsigned)(a.n_tokens + 3) / 4, 256, 0, st, a);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
    return a.p.d == 128 ? launch<__nv_bfloat16, 128>(a, st) : launch<__nv_bfloat16, 64>(a, st);
}

cudaError_t append_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
