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
#include <climits>

#include "lola_attn.cuh"

namespace lola {
namespace {

__device__ int32_t g_status;

constexpr int kLowPower = 27, kTopPower = 246;   // a quantised row's power of two, biased by 127: 2^-100 .. 2^119
constexpr int kFew = 760;   // tokens up to which a CTA takes one (five CTAs per SM)

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
    uint8_t* power;      // a row to be quantised (dst: its bytes): where its power of two goes; else null
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
    n.power = nullptr;
    n.x = *reinterpret_cast<const uint4*>(src + n.c0);
    n.y = *reinterpret_cast<const uint4*>(src + n.c1);
}
template <int VN>
__device__ __forceinline__ void turn_unit(float (&a)[VN], float (&b)[VN], const float4* cs, bool neighbours, int step) {
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
        const float4 c = cs[i * step];
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
}
template <typename T>
__device__ __forceinline__ void finish_unit(Unit<T>& n, bool neighbours, int step) {
    constexpr int VN = 16 / sizeof(T);
    if (n.cs) {
        float a[VN], b[VN];
        unpack<T>(n.x, a);
        unpack<T>(n.y, b);
        turn_unit<VN>(a, b, n.cs, neighbours, step);
        n.x = pack<T>(a);
        n.y = pack<T>(b);
    }
    *reinterpret_cast<uint4*>(n.dst + n.c0) = n.x;
    *reinterpret_cast<uint4*>(n.dst + n.c1) = n.y;
}

// A unit of a row that is quantised: its UH units are in as many neighbouring lanes (all lanes of the warp come
// here, those without a unit, `in` false, without effect).  The row's power of two is the smallest 2^e whose 448-fold
// reaches its largest magnitude: 448 = 1.75 2^8, so that e is the magnitude's own exponent - 8, and one more behind 1.75;
// it is kept in [-100, 119], where code 2^e is exact in bfloat16 and float32 and sums of 2^-e stay in float32.  A
// rotated key is not rounded before that.  Numbers that are not finite become the code for NaN, and do not count for e.
template <int VN, int UH>
__device__ __forceinline__ void store_codes(float (&a)[VN], float (&b)[VN], bool in, uint8_t* dst, int c0, int c1, uint8_t* to, bool first) {
    float top = 0.f;
    if (in) {
#pragma unroll
        for (int i = 0; i < VN; ++i) top = fmaxf(fmaxf(top, fabsf(a[i])), fabsf(b[i]));      // (NaN does not count)
    }
#pragma unroll
    for (int o = UH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (__any_sync(0xffffffffu, top == INFINITY)) {
        // infinities somewhere: they become NaN, which the conversion keeps
        top = 0.f;
        if (in) {
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                a[i] = fabsf(a[i]) < INFINITY ? a[i] : NAN;
                b[i] = fabsf(b[i]) < INFINITY ? b[i] : NAN;
                top = fmaxf(fmaxf(top, fabsf(a[i])), fabsf(b[i]));
            }
        }
#pragma unroll
        for (int o = UH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (!in) return;
    const uint32_t bits = __float_as_uint(top);
    const int power = min(max((int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u), kLowPower), kTopPower);
    const float down = __uint_as_float((uint32_t)(254 - power) << 23);
    auto codes = [&](const float(&v)[VN], uint32_t(&w)[VN / 4]) {
#pragma unroll
        for (int i = 0; i < VN / 4; ++i) {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * i + 1] * down), "f"(v[4 * i] * down));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * i + 3] * down), "f"(v[4 * i + 2] * down));
            w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
    };
    uint32_t x[VN / 4], y[VN / 4];
    codes(a, x);
    codes(b, y);
    if constexpr (VN == 8) {
        if (c1 == c0 + VN) {
            *reinterpret_cast<uint4*>(dst + c0) = make_uint4(x[0], x[1], y[0], y[1]);
        } else {
            *reinterpret_cast<uint2*>(dst + c0) = make_uint2(x[0], x[1]);
            *reinterpret_cast<uint2*>(dst + c1) = make_uint2(y[0], y[1]);
        }
    } else {
        *reinterpret_cast<uint32_t*>(dst + c0) = x[0];
        *reinterpret_cast<uint32_t*>(dst + c1) = y[0];
    }
    if (first) *to = (uint8_t)power;
}
template <typename T, int UH>
__device__ __forceinline__ void quantise_unit(Unit<T>& n, bool neighbours, int step, bool first) {
    constexpr int VN = 16 / sizeof(T);
    float a[VN], b[VN];
    if (n.power) {
        unpack<T>(n.x, a);
        unpack<T>(n.y, b);
        if (n.cs) turn_unit<VN>(a, b, n.cs, neighbours, step);
    }
    store_codes<VN, UH>(a, b, n.power != nullptr, reinterpret_cast<uint8_t*>(n.dst), n.c0, n.c1, n.power, first);
}

// Slot of token t (-1: no page, -2: no token of a sequence) and its position; one warp, valid in lane 0.
__device__ __forceinline__ int64_t find_slot(const AppendArgs& a, int t, int lane, int* position) {
    const PagedArgs& p = a.p;
    int b = t;
    int64_t pos, s = -2;
    if (a.cu_new) {
        b = warp_find_seq(a.cu_new, p.n_seq, t, lane);
        pos = b < 0 ? -1 : (int64_t)p.kv_len[b] - a.cu_new[b + 1] + t;
    } else {
        pos = (int64_t)p.kv_len[b] - 1;
    }
    if (lane == 0) {
        if (pos >= 0) {
            const int page = pos < paged_tokens(p, p.kv_len[b]) ? paged_page(p, b, pos) : -1;
            s = page < 0 ? -1 : paged_offset(p, page, 0, pos);
            if (page < 0) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
        }
        *position = a.positions ? a.positions[t] : (int)pos;
    }
    return s;
}
// The turn of one position at frequency f: its fraction, 2^-64.
__device__ __forceinline__ uint64_t turn_of(const AppendArgs& a, int f) {
    double turns = (double)a.inv_freq[f] * 0.15915494309189535;    // w / 2 pi
    turns -= floor(turns);
    return (uint64_t)(turns * 18446744073709551616.0);
}
// Cosine and sine of x turns (2^-64).
__device__ __forceinline__ float2 cos_sin(uint64_t x) {
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
    return make_float2(c, s);
}

// Slots, positions and cosines of the CTA's tokens t0 .. t0 + nt - 1 (all threads).
template <typename T, int D, int TOK, int NT>
__device__ __forceinline__ void place_tokens(const AppendArgs& a, int t0, int nt, float4 (&cs)[TOK][D / 4], uint64_t (&turn_sm)[D / 2],
                                             int64_t (&slot)[TOK], int (&pos_sm)[TOK], int rot) {
    constexpr int VN = 16 / sizeof(T);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const PagedArgs& p = a.p;

    for (int i = warp; i < nt; i += NT / kWarp) {
        int pos;
        const int64_t x = find_slot(a, t0 + i, lane, &pos);
        if (lane == 0) {
            slot[i] = x;
            pos_sm[i] = pos;
        }
    }
    // the turn of one position, by the last warps (the first ones look the tokens up)
    for (int f = NT - 1 - (int)threadIdx.x; f < rot / 2; f += NT) turn_sm[f] = turn_of(a, f);
    __syncthreads();
    const int ru = rot / (2 * VN);
    for (int e = threadIdx.x; e < nt * (rot / 2); e += NT) {
        const int i = TOK == 1 ? 0 : e / (rot / 2), f = e - i * (rot / 2);
        const float2 y = cos_sin(turn_sm[f] * (uint64_t)(int64_t)pos_sm[i]);    // modulo one turn
        reinterpret_cast<float2*>(cs[i])[((f % VN / 2) * ru + f / VN) * 2 + (f & 1)] = y;
    }
    __syncthreads();
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
    const PagedArgs& p = a.p;
    wait_for_last_kernel();
    const int rot = a.inv_freq ? a.rot : 0, ru = rot / (2 * VN);
    place_tokens<T, D, TOK, NT>(a, t0, nt, cs, turn_sm, slot, pos_sm, rot);
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

// Token t's rows, up to `most` lines of them, into L2, by threads i, i + step, ...
template <typename T, int D> __device__ __forceinline__ void prefetch_rows(const AppendArgs& a, int64_t t, int i, int step, int most) {
    constexpr int LN = D * sizeof(T) / 128;                                    // 128-byte lines of a head
    const int hq = a.Q.data ? a.p.Hq : 0, Hkv = a.p.Hkv;
    for (int e = i; e < min(most, (hq + 2 * Hkv) * LN); e += step) {
        const int l = e % LN, h = e / LN, hk = h - hq;
        const Rows& r = h < hq ? a.Q : hk >= Hkv ? a.V : a.K;
        const char* at = r.data + (t * r.row + (int64_t)(h < hq ? h : hk >= Hkv ? hk - Hkv : hk) * r.head) * (int)sizeof(T) + 128 * l;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
    }
}

// The same into a quantised cache, one token a CTA.
template <typename T, int D, int NT, int IN>
__global__ void __launch_bounds__(NT) quant_append_kernel(const AppendArgs a) {
    __shared__ __align__(16) float4 cs[1][D / 4];
    __shared__ uint64_t turn_sm[D / 2];
    __shared__ int64_t slot[1];
    __shared__ int pos_sm[1];
    constexpr int VN = 16 / sizeof(T), UH = D / (2 * VN);   // units per head
    const int t = blockIdx.x, lane = threadIdx.x % kWarp;
    const PagedArgs& p = a.p;
    wait_for_last_kernel();
    const int hq = a.Q.data ? p.Hq : 0, rot = a.inv_freq ? a.rot : 0, ru = rot / (2 * VN);
    // (the rows are on their way while position, page and cosines are found)
    prefetch_rows<T, D>(a, t, threadIdx.x, NT, INT_MAX);
    place_tokens<T, D, 1, NT>(a, t, 1, cs, turn_sm, slot, pos_sm, rot);
    const int64_t s = slot[0];
    if (s == -2) return;
    const bool nb = a.pairs == LOLA_PAIRS_NEIGHBOURS;
    const int units = (hq + (s < 0 ? 0 : 2 * p.Hkv)) * UH;
    for (int e0 = threadIdx.x; e0 - lane < units; e0 += NT * IN) {
        Unit<T> n[IN];
#pragma unroll
        for (int x = 0; x < IN; ++x) {
            const int e = e0 + x * NT, u = e % UH, h = e / UH;
            n[x].dst = nullptr;
            n[x].power = nullptr;
            if (e >= units) continue;
            if (h < hq) {
                load_unit<T>(n[x], reinterpret_cast<const T*>(a.Q.data) + t * a.Q.row + h * a.Q.head,
                             reinterpret_cast<T*>(a.QO.data) + t * a.QO.row + h * a.QO.head, u, rot, nb, cs[0]);
            } else {
                const bool v = h >= hq + p.Hkv;
                const int hk = h - hq - (v ? p.Hkv : 0);
                const Rows& r = v ? a.V : a.K;
                const int64_t at = s + (int64_t)hk * p.page * D;
                load_unit<T>(n[x], reinterpret_cast<const T*>(r.data) + t * r.row + hk * r.head,
                             reinterpret_cast<T*>((v ? p.V : p.K) + at), u, v ? 0 : rot, nb, cs[0]);
                n[x].power = (v ? p.Vs : p.Ks) + at / D;
            }
        }
#pragma unroll
        for (int x = 0; x < IN; ++x) {
            quantise_unit<T, UH>(n[x], nb, ru, (e0 + x * NT) % UH == 0);
            if (n[x].dst && !n[x].power) finish_unit<T>(n[x], nb, ru);
        }
    }
}

// Many tokens: a warp each.  A lane has the same unit of every head, and the unit's cosines and sines in registers (read
// from shared memory for every unit, two tokens a CTA, they took 15 us of 79).  IN units are under way.
// Bound by HBM bytes: 18 k tokens of 32/8 heads, d = 128, page 16: bfloat16 64 us, 6.3 TB/s, 94 % of the measured copy rate
// (two units and eight CTAs an SM 72); float32 121 us.
constexpr int kRowWarps = 4;
constexpr int kLines = 64;   // of a token, fetched ahead (all lines of float32 rows: 147 us, they leave L2 before they are read)
template <typename T, int D, int IN>
__global__ void __launch_bounds__(kRowWarps * kWarp, 5) quant_append_rows_kernel(const AppendArgs a) {
    constexpr int VN = 16 / sizeof(T), UH = D / (2 * VN), HS = kWarp / UH;     // units of a head, heads side by side
    constexpr int PP = D / 2 / kWarp;                                          // pairs whose angle a lane takes
    __shared__ uint64_t turn_sm[D / 2];
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, u = lane % UH, hs = lane / UH;
    const int64_t t = (int64_t)blockIdx.x * kRowWarps + warp;
    const PagedArgs& p = a.p;
    const int hq = a.Q.data ? p.Hq : 0, rot = a.inv_freq ? a.rot : 0;
    const bool nb = a.pairs == LOLA_PAIRS_NEIGHBOURS, turn = u < rot / (2 * VN), apart = turn && !nb;
    const int c0 = apart ? u * VN : u * 2 * VN, c1 = apart ? c0 + rot / 2 : c0 + VN;
    wait_for_last_kernel();
    if (t < a.n_tokens) prefetch_rows<T, D>(a, t, lane, kWarp, kLines);
    for (int f = threadIdx.x; f < rot / 2; f += kRowWarps * kWarp) turn_sm[f] = turn_of(a, f);
    int pos = 0;
    int64_t slot = t < a.n_tokens ? find_slot(a, (int)t, lane, &pos) : -2;
    __syncthreads();
    slot = __shfl_sync(0xffffffffu, slot, 0);
    pos = __shfl_sync(0xffffffffu, pos, 0);
    if (slot == -2) return;
    float co[VN], si[VN];
    {
        float2 mine[PP];
#pragma unroll
        for (int y = 0; y < PP; ++y) {
            const int f = lane * PP + y;
            mine[y] = f < rot / 2 ? cos_sin(turn_sm[f] * (uint64_t)(int64_t)pos) : make_float2(1.f, 0.f);
        }
#pragma unroll
        for (int z = 0; z < VN; ++z) {                                         // pair u VN + z
            co[z] = __shfl_sync(0xffffffffu, mine[z % PP].x, u * VN / PP + z / PP);
            si[z] = __shfl_sync(0xffffffffu, mine[z % PP].y, u * VN / PP + z / PP);
        }
    }
    auto turned = [&](float(&x)[VN], float(&y)[VN]) {
        auto pair = [](float& x, float& y, float co, float si) {
            const float x0 = x;
            x = x0 * co - y * si;
            y = y * co + x0 * si;
        };
        if (nb) {
#pragma unroll
            for (int z = 0; z < VN; ++z) {
                float(&w)[VN] = 2 * z < VN ? x : y;
                pair(w[2 * z % VN], w[2 * z % VN + 1], co[z], si[z]);
            }
        } else {
#pragma unroll
            for (int z = 0; z < VN; ++z) pair(x[z], y[z], co[z], si[z]);
        }
    };
    for (int h0 = 0; h0 < hq; h0 += HS * IN) {
        uint4 x[IN], y[IN];
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            if (h0 + HS * i >= hq) break;
            const int h = min(h0 + HS * i + hs, hq - 1);
            const T* src = reinterpret_cast<const T*>(a.Q.data) + t * a.Q.row + (int64_t)h * a.Q.head;
            x[i] = *reinterpret_cast<const uint4*>(src + c0);
            y[i] = *reinterpret_cast<const uint4*>(src + c1);
        }
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            const int h = h0 + HS * i + hs;
            if (h >= hq) break;
            if (turn) {
                float v[VN], w[VN];
                unpack<T>(x[i], v);
                unpack<T>(y[i], w);
                turned(v, w);
                x[i] = pack<T>(v);
                y[i] = pack<T>(w);
            }
            T* dst = reinterpret_cast<T*>(a.QO.data) + t * a.QO.row + (int64_t)h * a.QO.head;
            *reinterpret_cast<uint4*>(dst + c0) = x[i];
            *reinterpret_cast<uint4*>(dst + c1) = y[i];
        }
    }
    if (slot < 0) return;
    const int heads = 2 * p.Hkv;
    for (int h0 = 0; h0 < heads; h0 += HS * IN) {
        uint4 x[IN], y[IN];
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            if (h0 + HS * i >= heads) break;
            const int h = min(h0 + HS * i + hs, heads - 1);
            const bool v = h >= p.Hkv;
            const Rows& r = v ? a.V : a.K;
            const T* src = reinterpret_cast<const T*>(r.data) + t * r.row + (int64_t)(h - (v ? p.Hkv : 0)) * r.head;
            // (values are not rotated: the lane's chunks lie side by side)
            x[i] = *reinterpret_cast<const uint4*>(src + (v ? u * 2 * VN : c0));
            y[i] = *reinterpret_cast<const uint4*>(src + (v ? u * 2 * VN + VN : c1));
        }
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            if (h0 + HS * i >= heads) break;
            const int h = h0 + HS * i + hs;
            const bool v = h >= p.Hkv;
            float b[VN], c[VN];
            unpack<T>(x[i], b);
            unpack<T>(y[i], c);
            if (turn && !v) turned(b, c);
            const int64_t at = slot + (int64_t)(h - (v ? p.Hkv : 0)) * p.page * D;
            store_codes<VN, UH>(b, c, h < heads, reinterpret_cast<uint8_t*>(v ? p.V : p.K) + at, v ? u * 2 * VN : c0, v ? u * 2 * VN + VN : c1,
                                (v ? p.Vs : p.Ks) + at / D, u == 0);
        }
    }
}

// Few tokens: one a CTA, so that none waits for another's page lookup; many: four, whose rows of a head
// lie side by side in the page (512 tokens, 32/8 heads: 4.5 us one a CTA, 5.5 us four; 1024: 7.4 and 6.6).
// Into a quantised cache a warp each (512 tokens: 5 us one a CTA, 6 us a warp each; 1024: 8.3 and 7.8).
template <typename T, int D, bool QZ>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
    if constexpr (QZ) {
        if (a.n_tokens <= kFew) return launch_behind(quant_append_kernel<T, D, 128, 3>, (unsigned)a.n_tokens, 128, 0, st, a);
        return launch_behind(quant_append_rows_kernel<T, D, 4>, ((unsigned)a.n_tokens + kRowWarps - 1) / kRowWarps, kRowWarps * kWarp, 0, st, a);
    } else {
        if (a.n_tokens <= kFew) return launch_behind(paged_append_kernel<T, D, 1, 128, 3>, (unsigned)a.n_tokens, 128, 0, st, a);
        return launch_behind(paged_append_kernel<T, D, 4, 256, 3>, (unsigned)(a.n_tokens + 3) / 4, 256, 0, st, a);
    }
}
template <typename T>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
    if (a.p.Ks) return a.p.d == 128 ? launch<T, 128, true>(a, st) : launch<T, 64, true>(a, st);
    return a.p.d == 128 ? launch<T, 128, false>(a, st) : launch<T, 64, false>(a, st);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t st) {
    return a.p.dtype == LOLA_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

cudaError_t append_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
