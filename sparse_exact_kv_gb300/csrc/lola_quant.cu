// K11: the quantised paged cache, read back as rows and by single tokens.
//
// A row (a token's key or value of one head) is kept as e4m3 numbers and one power of two:
// x_i ~ code_i 2^e, both exact in bfloat16 and float32 (lola_append.cu writes them).
//
// Attention (o = sum_j p_j v_j / sum_j p_j over the kv_len tokens of a sequence) is K10's: equal pieces of the
// whole batch for every SM, a producer warp with a ring of tiles, a running softmax per warp, the pieces' join.
// Here the codes become float16 numbers (exact) in the registers and go to the warps' float16 products; the
// powers of two of the keys scale the scores, those of the values join the weights in the exponent:
//   s_j = c 2^{e_j} q . code_j,   w_j = 2^{s_j + f_j - m},   O = sum_j w_j code'_j,   l = sum_j w_j 2^{-f_j},
// m set above the largest s_j + f_j: everything but the exponentials, the weights' rounding and the sums is exact.
// q comes as float16 numbers of its row's own power of two (its largest number in [2^14, 2^15): a bfloat16 number
// loses nothing down to 2^-28 of that; a float32 number is kept in two parts, to 2^-39 of it), the weights as
// float16 numbers of 2^15 w_j (rounded by 2^-12 of themselves, or by 2^-40 where they are small; float32 io: two parts).
// The contraction's channels may come in any order: a lane's four neighbouring codes of K, one word, are its four
// channels of a product, and the same four of q.  A word of V holds two channels of two tokens and is permuted first.
#include "lola_codes.cuh"
#include "lola_paged.cuh"

namespace lola {
namespace {

__device__ __forceinline__ void mma16816_h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// what the float16 numbers of x and y leave
__device__ __forceinline__ uint32_t half2_rest(float x, float y, uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return half2_of(x - f.x, y - f.y);
}
template <typename TO, int D, bool HALF> struct QSmem {
    static constexpr int NW = kCons / kWarp;
    static constexpr int HR = HALF ? 1 : 2, R8 = 8 * HR, CK = 512 / R8;     // rows kept; columns joined at a time
    static constexpr int kPitch = D * (int)sizeof(TO) + 16;                 // Q rows
    float red[NW][R8][CK];
    float ms[NW][R8], ls[NW][R8];
    uint8_t q[2][kRows * kPitch];
};

// All eight warps on a segment, in two groups that take its tiles in turn; a warp has 16 of a tile's 64 tokens.
// HALF: at most 8 query rows (rows 8-15 of the products hold anything and are left alone).  TO: q and o.
template <typename TO, int D, bool HALF, bool SH>
__global__ void __launch_bounds__(kThreads, 1) quant_decode_kernel(const __grid_constant__ Maps maps, const Args a) {
    using T = uint8_t;
    using C = Cfg<T, D>;
    using M = QSmem<TO, D, HALF>;
    constexpr int HR = M::HR, CK = M::CK, NW = M::NW, NT = kCons;
    constexpr bool kTwo = sizeof(TO) == 4;                             // q and the weights in two parts
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    __shared__ __align__(16) M x;
    __shared__ __align__(8) Bars<C::kStages> bars;
    __shared__ uint32_t bad_sm[C::kStages];
    __shared__ int abort_sm, go;
    __shared__ Seg segs[2];
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 1);
            mbar_init(smem_u32(&bars.empty[s]), 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars.seg_full[s]), 1);
            mbar_init(smem_u32(&bars.seg_empty[s]), NW);
        }
        abort_sm = 0;
        bars.issued = bars.given = bars.arrived[0] = bars.arrived[1] = 0;
    }
    wait_for_last_kernel();
    Start st;
    if (!find_start<SH>(a, &st)) return;
    if (warp == NW) produce<T, TO, D, 2, SH>(maps, a, st, sb, smem_u32(x.q[0]), M::kPitch, bars, segs, bad_sm, &abort_sm, lane);
    const int grp = warp >> 2, k0 = (warp & 3) * 16, g8 = lane >> 2, q4 = lane & 3, q2 = q4 * 2;
    auto bar = [&] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    const int box = min(p.page, kTile), lb = 31 - __clz(box);
    // 16-byte chunk ch of token k's row: rows of 128 bytes (two tokens at d = 64), chunks swizzled
    auto chunk_at = [](int k, int ch) {
        const int row = k * D / 128, c = D == 128 ? ch : (k & 1) * 4 + ch;
        return (uint32_t)(row * 128 + (((c ^ row) & 7) << 4));
    };
    const int token = k0 + ((lane >> 3) & 1) * 8 + (lane & 7), ch0 = lane >> 4;     // this lane's ldmatrix row
    for (int i = 0; warp < NW; ++i) {
        const int slot = i & 1;
        if (group_or<NT>(1, !ring_wait(smem_u32(&bars.seg_full[slot]), (uint32_t)(i >> 1) & 1, &abort_sm))) {
            if (tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
        const Seg g = segs[slot];
        if (g.R < 0) break;
        if (!SH && !g.whole && tid == 64) open_cells<D>(a, g);
        // ---- q: rows g8 and g8 + 8, channels 16 y + 4 q4 .. + 3, with a power of two of the row's own ----
        uint32_t qa[D / 16][4], qr[kTwo ? D / 16 : 1][4];
        float qs[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint8_t* row = x.q[slot] + (g8 + 8 * r) * M::kPitch;
            float v[D / 16][4];
            uint32_t top = 0u;
#pragma unroll
            for (int y = 0; y < D / 16; ++y) {
                if constexpr (kTwo) {
                    const float4 z = *reinterpret_cast<const float4*>(row + (16 * y + 4 * q4) * 4);
                    v[y][0] = z.x, v[y][1] = z.y, v[y][2] = z.z, v[y][3] = z.w;
                } else {
                    const uint2 z = *reinterpret_cast<const uint2*>(row + (16 * y + 4 * q4) * 2);
                    v[y][0] = __uint_as_float(z.x << 16), v[y][1] = __uint_as_float(z.x & 0xffff0000u);
                    v[y][2] = __uint_as_float(z.y << 16), v[y][3] = __uint_as_float(z.y & 0xffff0000u);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[y][e]) & 0x7fffffffu);
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t up = min(268u - (top >> 23), 240u);         // the largest magnitude goes to [2^14, 2^15)
            const float f = __uint_as_float(up << 23);
            qs[r] = a.scale_log2 * __uint_as_float((254u - up) << 23);
#pragma unroll
            for (int y = 0; y < D / 16; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float u = v[y][2 * e] * f, w = v[y][2 * e + 1] * f;
                    qa[y][2 * e + r] = half2_of(u, w);
                    if constexpr (kTwo) qr[y][2 * e + r] = half2_rest(u, w, qa[y][2 * e + r]);
                }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive1(smem_u32(&bars.seg_empty[slot]));   // (g and the Q rows are in registers)
        float o[D / 16][2][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int y = 0; y < D / 16; ++y)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[y][e >> 2][e & 3] = 0.f;
        bool ok = true;
        for (int t = (g.n0 ^ grp) & 1; t < g.tiles; t += 2) {
            const int n = g.n0 + t, s = n % C::kStages;
            ok = issued_wait(&bars.issued, n, &abort_sm) &&
                 ring_wait(smem_u32(&bars.full[s]), (uint32_t)(n / C::kStages) & 1, &abort_sm);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t kt = sb + (uint32_t)s * 2 * C::kHalf, vt = kt + C::kHalf;
            const uint8_t* powers = sm + (size_t)C::kStages * 2 * C::kHalf + (size_t)s * C::kScales + k0 + q2;
            const int left = g.len - t * kTile;
            const uint32_t bad = bad_sm[s];
            // ---- S: 16 rows x 16 tokens, two chains a token half ----
            float c0[2][4] = {}, c1[2][4] = {};
#pragma unroll
            for (int y = 0; y < D / 32; ++y) {
                uint32_t kb[4];
                ldsm4(kt + chunk_at(token, 2 * y + ch0), kb);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    uint32_t lo, hi;
                    widen(kb[z], lo, hi);
                    mma16816_h(z >> 1 ? c1[z & 1] : c0[z & 1], qa[2 * y + (z >> 1)], lo, hi);
                    if constexpr (kTwo) mma16816_h(z >> 1 ? c1[z & 1] : c0[z & 1], qr[2 * y + (z >> 1)], lo, hi);
                }
            }
            // ---- scores and exponents of the weights: tokens k0 + q2, + 1, + 8, + 9 ----
            float sc[2][4], down[2][2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t kp = *reinterpret_cast<const uint16_t*>(powers + 8 * y), vp = *reinterpret_cast<const uint16_t*>(powers + kTile + 8 * y);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint32_t kb = z ? kp >> 8 : kp & 255u, vb = z ? vp >> 8 : vp & 255u;
                    const float fk = __uint_as_float(kb << 23), fv = (float)(int)vb - 127.f;
                    down[y][z] = power_down(vb);
#pragma unroll
                    for (int r = 0; r < HR; ++r) sc[y][2 * r + z] = fmaf((c0[y][2 * r + z] + c1[y][2 * r + z]) * qs[r], fk, fv);
                }
            }
            if (left < k0 + 16 || bad) {
                // tokens behind the sequence or on bad pages: no score, and their V rows (which may
                // hold anything) become zero
                const int nk = max(0, min(kTile, left));
                auto hidden = [&](int k) { return k >= nk || ((bad >> (k >> lb)) & 1u); };
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 2 * HR; ++e)
                        if (hidden(k0 + 8 * y + q2 + (e & 1))) sc[y][e] = -INFINITY;
                for (int k = k0; k < k0 + 16; ++k)
                    if (hidden(k) && lane < D / 16)
                        *reinterpret_cast<uint4*>(sm + (size_t)s * 2 * C::kHalf + C::kHalf + chunk_at(k, lane)) = make_uint4(0, 0, 0, 0);
                fence_async_smem();            // (before the ring's next copy lands on these rows)
                __syncwarp();
            }
            // ---- running maximum, weights ----
            uint32_t pa[4] = {0u, 0u, 0u, 0u}, pr[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int r = 0; r < HR; ++r) {
                float bm = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                const float top = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2)) + kRaise;
                const bool need = top > m[r] + kRaise;
                if (__any_sync(0xffffffffu, need)) {
                    const float f = need ? ex2(m[r] - top) : 1.f;
                    if (need) m[r] = top;
                    l[r] *= f;
#pragma unroll
                    for (int y = 0; y < D / 16; ++y)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            o[y][e][2 * r] *= f;
                            o[y][e][2 * r + 1] *= f;
                        }
                }
                const float base = m[r] == -INFINITY ? 0.f : m[r];
                float w[2][2];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        w[y][z] = ex2(sc[y][2 * r + z] - base);
                        l[r] = fmaf(w[y][z], down[y][z], l[r]);
                        w[y][z] *= kUp;
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    pa[2 * y + r] = half2_of(w[y][0], w[y][1]);
                    if constexpr (kTwo) pr[2 * y + r] = half2_rest(w[y][0], w[y][1], pa[2 * y + r]);
                }
            }
            // ---- O += P V ----
#pragma unroll
            for (int y = 0; y < D / 32; ++y) {
                uint32_t vb[4];
                ldsm4_t(vt + chunk_at(token, 2 * y + ch0), vb);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t e0, o0, e1, o1;
                    widen(__byte_perm(vb[2 * z], 0u, 0x3120), e0, o0);
                    widen(__byte_perm(vb[2 * z + 1], 0u, 0x3120), e1, o1);
                    mma16816_h(o[2 * y + z][0], pa, e0, e1);
                    mma16816_h(o[2 * y + z][1], pa, o0, o1);
                    if constexpr (kTwo) {
                        mma16816_h(o[2 * y + z][0], pr, e0, e1);
                        mma16816_h(o[2 * y + z][1], pr, o0, o1);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(smem_u32(&bars.empty[s]));
        }
        // ---- the segment's end: add the warps in order, then o or the piece's record ----
        if (group_or<NT>(1, !ok)) {
            if (tid == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (q4 == 0) {
                x.ms[warp][g8 + 8 * r] = m[r];
                x.ls[warp][g8 + 8 * r] = l[r];
            }
        }
        bar();
        float f[2];
#pragma unroll
        for (int r = 0; r < HR; ++r) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < NW; ++w) mm = fmaxf(mm, x.ms[w][g8 + 8 * r]);
            f[r] = ex2(m[r] - (mm == -INFINITY ? 0.f : mm)) * (1.f / kUp);
        }
        float* rec = segment_record<D, SH>(a, g);
        const int er = 4 * (tid & 127) / CK, ec = 4 * (tid & 127) % CK;        // 128 threads x 4 columns = R8 x CK
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, x.ms[w][er]);
#pragma unroll
        for (int w = 0; w < NW; ++w) ll = fmaf(x.ls[w][er], ex2(x.ms[w][er] - (mm == -INFINITY ? 0.f : mm)), ll);
#pragma unroll
        for (int c = 0; c < D; c += CK) {
            if (c > 0) bar();
#pragma unroll
            for (int y = 0; y < CK / 16; ++y)
#pragma unroll
                for (int r = 0; r < HR; ++r) {
                    const float(&z)[2][4] = o[c / 16 + y];
                    *reinterpret_cast<float4*>(&x.red[warp][g8 + 8 * r][16 * y + 4 * q4]) =
                        make_float4(z[0][2 * r] * f[r], z[1][2 * r] * f[r], z[0][2 * r + 1] * f[r], z[1][2 * r + 1] * f[r]);
                }
            bar();
            if (tid < 128) {
                float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float4 z = *reinterpret_cast<const float4*>(&x.red[w][er][ec]);
                    y[0] += z.x;
                    y[1] += z.y;
                    y[2] += z.z;
                    y[3] += z.w;
                }
                if (er < g.R) write_out<TO, D, SH>(a, g, g.whole, rec, er, c + ec, y, mm, ll);
            }
        }
        if (!SH && !g.whole) join_pieces<TO, D, NT>(a, g, tid, &go, bars.arrived, bar);
    }
    __syncthreads();
    if (abort_sm) settle<D, C::kStages, 2, SH>(a, bars);
}

template <typename TO, int D, bool SH>
cudaError_t launch_quant(const DecodeArgs& d, cudaStream_t st) {
    static std::atomic<uint64_t> done[2] = {};
    return !SH && d.p.G <= 8 ? launch_kernel<uint8_t, D>(quant_decode_kernel<TO, D, true, false>, done[0], d, st)
                             : launch_kernel<uint8_t, D>(quant_decode_kernel<TO, D, false, SH>, done[1], d, st);
}
template <bool SH> cudaError_t launch_quant(const DecodeArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_quant<float, 128, SH>(a, st) : launch_quant<float, 64, SH>(a, st);
    return a.p.d == 128 ? launch_quant<__nv_bfloat16, 128, SH>(a, st) : launch_quant<__nv_bfloat16, 64, SH>(a, st);
}

// ---- the cached rows as rows ----
// Row r of the packed output is a token of the sequence whose tokens, counted from the first sequence's on, hold
// number r.  Each CTA adds the lengths up for itself, looks its rows' pages up, and has NU units of 16 bytes of
// output in flight a thread.  Bound by bytes: each code read once, each number written once.
constexpr int kReadRows = 32, kReadThreads = 256;

template <typename T> __device__ __forceinline__ uint4 read_unit(const uint8_t* src, float f);
template <> __device__ __forceinline__ uint4 read_unit<float>(const uint8_t* src, float f) {
    uint32_t lo, hi;
    widen(*reinterpret_cast<const uint32_t*>(src), lo, hi);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_uint4(__float_as_uint(x.x * f), __float_as_uint(x.y * f), __float_as_uint(y.x * f), __float_as_uint(y.y * f));
}
template <> __device__ __forceinline__ uint4 read_unit<__nv_bfloat16>(const uint8_t* src, float f) {
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t lo, hi;
        widen(i ? w.y : w.x, lo, hi);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        r[2 * i] = pack2(x.x * f, x.y * f);
        r[2 * i + 1] = pack2(y.x * f, y.y * f);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) quant_read_kernel(const ReadArgs a) {
    constexpr int VN = 16 / sizeof(T), UH = D / VN;                    // numbers of a unit, units of a head
    __shared__ int64_t sums[kReadThreads / kWarp];
    __shared__ int64_t from[kReadRows];                                // (page, slot) of a row: -1 zeros, -2 no row
    const PagedArgs& p = a.p;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const int64_t r0 = (int64_t)blockIdx.x * kReadRows, r1 = min(r0 + kReadRows, (int64_t)a.total);
    wait_for_last_kernel();
    if (threadIdx.x < kReadRows) from[threadIdx.x] = -2;
    int64_t before = 0;
    int bits = 0;
    for (int base = 0; base < p.n_seq; base += kReadThreads) {
        const int b = base + threadIdx.x;
        const int len = b < p.n_seq ? p.kv_len[b] : 0;
        const int64_t n = b < p.n_seq ? paged_tokens(p, len) : 0;
        if (len > n && len > 0) bits |= LOLA_ATTN_BAD_PAGE;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == kWarp - 1) sums[warp] = inc;
        __syncthreads();
        int64_t pre = before, all = before;
#pragma unroll
        for (int w = 0; w < kReadThreads / kWarp; ++w) {
            if (w < warp) pre += sums[w];
            all += sums[w];
        }
        const int64_t hi = pre + inc, lo = hi - n;
        if (blockIdx.x == 0 && b < p.n_seq) {
            a.cu[b + 1] = (int)min(hi, (int64_t)a.total);
            if (b == 0) a.cu[0] = 0;
            if (hi > a.total) bits |= LOLA_ATTN_BAD_OFFSETS;
        }
        for (int64_t r = max(lo, r0); r < min(hi, r1); ++r) {
            const int64_t pos = r - lo;
            const int page = paged_page(p, b, pos);
            if (page < 0) bits |= LOLA_ATTN_BAD_PAGE;
            from[r - r0] = page < 0 ? -1 : (int64_t)page * p.Hkv * p.page + (pos & (p.page - 1));
        }
        before = all;
        if (blockIdx.x > 0 && before >= r1) break;
    }
    if (bits) atomicOr(&g_status, bits);
    __syncthreads();
    constexpr int NU = 8;
    const int units = kReadRows * p.Hkv * UH;
    for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* pool = reinterpret_cast<const uint8_t*>(kv ? p.V : p.K);
        const uint8_t* powers = kv ? p.Vs : p.Ks;
        const Rows& out = kv ? a.V : a.K;
        for (int e0 = threadIdx.x; e0 < units; e0 += NU * kReadThreads) {
            uint4 y[NU];
            T* dst[NU];
#pragma unroll
            for (int x = 0; x < NU; ++x) {
                const int e = e0 + x * kReadThreads, u = e % UH, rh = e / UH, i = rh / p.Hkv, h = rh - i * p.Hkv;
                dst[x] = nullptr;
                if (e >= units || from[i] == -2) continue;
                dst[x] = reinterpret_cast<T*>(out.data) + (r0 + i) * out.row + (int64_t)h * out.head + u * VN;
                y[x] = make_uint4(0, 0, 0, 0);
                if (from[i] < 0) continue;
                const int64_t row = from[i] + (int64_t)h * p.page;
                y[x] = read_unit<T>(pool + row * D + u * VN, __uint_as_float((uint32_t)powers[row] << 23));
            }
#pragma unroll
            for (int x = 0; x < NU; ++x)
                if (dst[x]) *reinterpret_cast<uint4*>(dst[x]) = y[x];
        }
    }
}
template <typename T, int D> cudaError_t launch_read(const ReadArgs& a, cudaStream_t st) {
    const unsigned grid = a.total > 0 ? (unsigned)((a.total + (int64_t)kReadRows - 1) / kReadRows) : 1u;
    return launch_behind(quant_read_kernel<T, D>, grid, kReadThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_quant_decode(const DecodeArgs& a, cudaStream_t st) { return launch_quant<false>(a, st); }
cudaError_t launch_quant_prefix(const DecodeArgs& a, cudaStream_t st) { return launch_quant<true>(a, st); }

cudaError_t launch_quant_read(const ReadArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_read<float, 128>(a, st) : launch_read<float, 64>(a, st);
    return a.p.d == 128 ? launch_read<__nv_bfloat16, 128>(a, st) : launch_read<__nv_bfloat16, 64>(a, st);
}

cudaError_t quant_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
