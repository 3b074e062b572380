// K11: the quantised paged cache, read back as rows and by single tokens.
//
// A row (a token's key or value of one head) is kept as e4m3 numbers and one power of two:
// x_i ~ code_i 2^e, both exact in bfloat16 and float32 (lola_append.cu writes them).
//
// Attention (o = sum_j p_j v_j / sum_j p_j over the kv_len tokens of a sequence) is K10's: equal pieces of the
// whole batch for every SM, a producer warp with a ring of tiles, a running softmax per warp, the pieces' join.
// Here the codes become float16 numbers (exact) in the registers and go to the warps' float16 products; the
// powers of two of the keys scale the scores, those of the values join the weights in the exponent:
//   s_j = c 2^{e_j} q . code_j,   w_j = 2^{s_j + f_j - m},   O = sum_j w_j code'_j,   l = sum_j 2^{s_j - r},
// m set above the largest s_j + f_j, r, a lane's own, above its largest s_j: everything but the exponentials, the weights'
// rounding and the sums is exact, however far the powers lie apart (l as a sum of w_j 2^{-f_j} lost rows whose power is
// 2^-110 of another's: of zeros, which have 2^-100, beside numbers of 2^20).  At a segment's end O comes to 2^{m - r}, r
// above all lanes' and with room for sums of large values (kRoom), and from there on m and l are the scores'.
// q comes as float16 numbers of its row's own power of two (its largest number in [2^14, 2^15): a bfloat16 number
// loses nothing down to 2^-28 of that; a float32 number is kept in two parts, to 2^-39 of it), the weights as
// float16 numbers of 2^15 w_j (rounded by 2^-12 of themselves, or by 2^-40 where they are small; float32 io: two parts).
// The products have tokens, then channels, as M and the query rows as N, eight at a time: S^T = K Q^T, O^T = V^T P^T, the
// weights turned by movmatrix in between.  Groups of up to eight query heads then cost half the products and registers
// of the other way round (M = 16 rows), which leaves room for twelve warps in place of eight.
// The contraction's channels may come in any order: a lane's four neighbouring codes of K, one word, are its four
// channels of a product, and the same four of q.  A word of V holds two channels of two tokens and is permuted first.
// Bound by reading codes and powers once.  Measured (bfloat16 io, d = 128): 64 sequences of 1000-8000 tokens, 32/8 heads,
// 90 us, 5.0 TB/s (loads alone, without products: 75 us; the rest is the segments' ends; l out of the weights: 88 us); 3 of
// 65536-131072 tokens, 40/8 heads, 98 us, 6.1 TB/s; one of 1000 tokens 9.3 us, a chain of dependent accesses as in K10.
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
// the 8 x 8 numbers of a warp's lanes (row lane / 4, columns 2 (lane % 4) and + 1), transposed
__device__ __forceinline__ uint32_t turned(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

constexpr float kNone = -3.0e38f;       // below any score (QZ: in place of an infinity, which differences would have to avoid)

// T: the cache's numbers (bfloat16, or uint8_t: e4m3).  NB: query rows in eights.
template <typename T, typename TO, int D, int NB> struct TSmem {
    static constexpr int kGroups = NB == 1 ? 3 : 2;                         // groups of four consumer warps
    static constexpr int NW = 4 * kGroups, kAll = NW + (sizeof(T) == 1 ? 3 : 1);    // consumer warps, and all
    static constexpr int NS = sizeof(TO) == 4 ? 2 : 4;                      // segments under way
    static constexpr int kRing = (D == 128 ? 5 : 10) - (NB == 1 ? 0 : D == 128 ? 1 : 2);   // tiles
    static constexpr int kCk = NB == 1 ? 64 : 32;                           // columns joined at a time
    static constexpr int kPitch = D * (int)sizeof(TO) + 16;                 // Q rows
    float red[kGroups][4][8 * NB][kCk + 8];                                 // (rows 32 bytes apart: 8-byte stores of four rows)
    float part[2][kGroups][8 * NB][D];                                      // the groups' parts of a segment
    float part_ml[2][kGroups][2][8 * NB];
    float ms[kGroups][4][8 * NB], ls[kGroups][4][8 * NB];
    uint8_t q[NS][8 * NB * kPitch];
};

// Tile n is group n % kGroups', a warp has a quarter of its tokens, 16 at a time.  A group that is done with its tiles of a
// segment adds its warps up and goes on to the next segment; the last of a segment's groups to be done adds the groups up, in
// their order.  So a sequence of one tile takes one group, and the others' tiles run beside its end (all warps at the segment's
// end together: 64 sequences of 1000-8000 tokens, 32/8 heads, d = 128, e4m3, 94 us, by turns 88; 1024 items of 64 tokens
// 37 and 18 us).
template <typename T, typename TO, int D, int NB, bool SH, bool PRE>
__global__ void __launch_bounds__(TSmem<T, TO, D, NB>::kAll * kWarp, 1) decode_t_kernel(const __grid_constant__ Maps maps, const Args a) {
    using M = TSmem<T, TO, D, NB>;
    using C = Ring<Cfg<T, D>, M::kRing>;
    constexpr int NW = M::NW, NT = 128, kGroups = M::kGroups, NS = M::NS, CK = M::kCk;
    constexpr bool QZ = sizeof(T) == 1, kTwo = sizeof(TO) == 4;        // kTwo: q and the weights in two parts
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    M& x = *reinterpret_cast<M*>(sm + C::kSmem - 1024);
    __shared__ __align__(8) Bars<C::kStages, NS> bars;
    __shared__ uint32_t bad_sm[C::kStages];
    __shared__ int abort_sm, go[kGroups];
    __shared__ int here[2], joined[2];                     // groups whose parts are in part[]; segments that were added up there
    __shared__ Seg segs[NS];
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), C::kFull);
            mbar_init(smem_u32(&bars.empty[s]), 4);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bars.seg_full[s]), 1);
            mbar_init(smem_u32(&bars.seg_empty[s]), NW);
        }
        abort_sm = here[0] = here[1] = joined[0] = joined[1] = 0;
        bars.issued = bars.ahead = bars.given = bars.arrived[0] = bars.arrived[1] = 0;
    }
    wait_for_last_kernel();
    Start st;
    if (!find_start<SH, M::kAll * kWarp, C::kTokens, kRows, PRE>(a, &st)) return;
    if (warp >= NW) produce<T, TO, D, NS, SH, C, 8 * NB, PRE>(maps, a, st, sb, smem_u32(x.q[0]), M::kPitch, bars, segs, bad_sm, &abort_sm, lane, warp - NW);
    const int grp = warp >> 2, w4 = warp & 3, gt = tid & 127, g8 = lane >> 2, q4 = lane & 3, q2 = q4 * 2;
    auto bar = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(NT) : "memory"); };
    const int box = min(p.page, C::kTokens), lb = 31 - __clz(box);
    // 16-byte chunk ch of token k's row: rows of 128 bytes, chunks swizzled; bfloat16: a box of 128-byte columns, e4m3: one
    // column, whose rows are two tokens at d = 64
    auto chunk_at = [&](int k, int ch) {
        if constexpr (QZ) {
            const int row = k * D / 128, c = D == 128 ? ch : (k & 1) * 4 + ch;
            return (uint32_t)(row * 128 + (((c ^ row) & 7) << 4));
        } else {
            return (uint32_t)((k >> lb) * box * C::kRowBytes + (k & (box - 1)) * 128 + (ch >> 3) * box * 128 + (((ch ^ k) & 7) << 4));
        }
    };
    // this lane's ldmatrix rows: of K, and of V (e4m3: the same)
    const int krow = ((lane >> 3) & 1) * 8 + (lane & 7), kch = lane >> 4;
    const int vrow = QZ ? krow : (lane >> 4) * 8 + (lane & 7), vch = QZ ? kch : (lane >> 3) & 1;
    int multi = 0;                                          // segments of several groups so far
    for (int i = 0; warp < NW; ++i) {
        const int slot = i % NS;
        if (group_or<NT>(1 + grp, !ring_wait(smem_u32(&bars.seg_full[slot]), (uint32_t)(i / NS) & 1, &abort_sm))) {
            if (gt == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
        const Seg g = segs[slot];
        if (g.R < 0) break;
        const int t0 = (grp + kGroups - g.n0 % kGroups) % kGroups, groups = min(kGroups, g.tiles), turn = multi;
        multi += groups > 1;
        if (t0 >= g.tiles) {                                            // (none of its tiles)
            __syncwarp();
            if (lane == 0) mbar_arrive1(smem_u32(&bars.seg_empty[slot]));
            continue;
        }
        if (!SH && !g.whole && t0 == 0 && gt == 64) open_cells<D>(a, g);
        // ---- q: row 8 b + g8.  e4m3: channels 16 y + 4 q4 .. + 3, with a power of two of the row's own; the lanes' rows of the
        // scores are 8 b + q2 and + 1.  bfloat16: channels 16 y + q2, + 1, + 8, + 9 ----
        uint32_t qa[NB][D / 16][2], qr[kTwo ? NB : 1][kTwo ? D / 16 : 1][2];
        float qs[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint8_t* row = x.q[slot] + (g8 + 8 * b) * M::kPitch;
            if constexpr (QZ) {
                uint32_t top = 0u;
                auto channels = [&](int y, float(&v)[4]) {
                    if constexpr (kTwo) {
                        const float4 z = *reinterpret_cast<const float4*>(row + (16 * y + 4 * q4) * 4);
                        v[0] = z.x, v[1] = z.y, v[2] = z.z, v[3] = z.w;
                    } else {
                        const uint2 z = *reinterpret_cast<const uint2*>(row + (16 * y + 4 * q4) * 2);
                        v[0] = __uint_as_float(z.x << 16), v[1] = __uint_as_float(z.x & 0xffff0000u);
                        v[2] = __uint_as_float(z.y << 16), v[3] = __uint_as_float(z.y & 0xffff0000u);
                    }
                };
#pragma unroll
                for (int y = 0; y < D / 16; ++y) {
                    float v[4];
                    channels(y, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t up = min(268u - (top >> 23), 240u);     // the largest magnitude goes to [2^14, 2^15)
                const float f = __uint_as_float(up << 23);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    qs[b][e] = a.scale_log2 * __uint_as_float((254u - __shfl_sync(0xffffffffu, up, 4 * (q2 + e))) << 23);
#pragma unroll
                for (int y = 0; y < D / 16; ++y) {
                    float v[4];
                    channels(y, v);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float u = v[2 * e] * f, w = v[2 * e + 1] * f;
                        qa[b][y][e] = half2_of(u, w);
                        if constexpr (kTwo) qr[b][y][e] = half2_rest(u, w, qa[b][y][e]);
                    }
                }
            } else {
#pragma unroll
                for (int y = 0; y < D / 16; ++y)
#pragma unroll
                    for (int e = 0; e < 2; ++e) qa[b][y][e] = *reinterpret_cast<const uint32_t*>(row + (16 * y + 8 * e + q2) * 2);
                qs[b][0] = qs[b][1] = a.scale_log2;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive1(smem_u32(&bars.seg_empty[slot]));   // (g and the Q rows are in registers)
        // o: channels 16 y + 2 g8 (0, 1) and + 1 (2, 3), or (bfloat16) + g8 and + 8 + g8; rows 8 b + q2 and + 1
        // ml: what l is kept against (QZ)
        float o[D / 16][NB][4], m[NB][2], l[NB][2];
        [[maybe_unused]] float ml[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[b][e] = ml[b][e] = QZ ? kNone : -INFINITY;
                l[b][e] = 0.f;
            }
#pragma unroll
            for (int y = 0; y < D / 16; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[y][b][e] = 0.f;
        }
        bool ok = true;
        for (int t = t0; t < g.tiles; t += kGroups) {
            const int n = g.n0 + t, s = n % C::kStages;
            ok = issued_wait(&bars.issued, n, &abort_sm) &&
                 ring_wait(smem_u32(&bars.full[s]), (uint32_t)(n / C::kStages) & 1, &abort_sm);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t kt = sb + (uint32_t)s * 2 * C::kHalf, vt = kt + C::kHalf;
            [[maybe_unused]] const uint8_t* powers = sm + (size_t)C::kStages * 2 * C::kHalf + (size_t)s * C::kScales + g8;
            const uint32_t info = bad_sm[s], bad = PRE ? info & 0xffffu : info;
            const int left = PRE ? (int)(info >> 16) : g.len - t * C::kTokens;
#pragma unroll 1
            for (int k0 = w4 * (C::kTokens / 4), end = k0 + C::kTokens / 4; k0 < end; k0 += 16) {
                // ---- S^T: 16 tokens x 8 rows, two chains ----
                float c0[NB][4] = {}, c1[NB][4] = {};
                if constexpr (QZ) {
#pragma unroll
                    for (int y = 0; y < D / 32; ++y) {
                        uint32_t kb[4];
                        ldsm4(kt + chunk_at(k0 + krow, 2 * y + kch), kb);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t ka[4];                            // tokens g8, g8 + 8: channels 4 q4, + 1; then + 2, + 3
                            widen(kb[2 * z], ka[0], ka[2]);
                            widen(kb[2 * z + 1], ka[1], ka[3]);
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                mma16816_h(z ? c1[b] : c0[b], ka, qa[b][2 * y + z][0], qa[b][2 * y + z][1]);
                                if constexpr (kTwo) mma16816_h(z ? c1[b] : c0[b], ka, qr[b][2 * y + z][0], qr[b][2 * y + z][1]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < D / 16; ++y) {
                        uint32_t ka[4];
                        ldsm4(kt + chunk_at(k0 + krow, 2 * y + kch), ka);
#pragma unroll
                        for (int b = 0; b < NB; ++b) mma16816(y & 1 ? c1[b] : c0[b], ka, qa[b][y][0], qa[b][y][1]);
                    }
                }
                // ---- scores, and (e4m3) what the weights' exponents have besides: tokens k0 + g8 (0, 1), + 8 (2, 3) ----
                float sc[NB][4], fv[2] = {0.f, 0.f};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float fk = 1.f;
                    if constexpr (QZ) {
                        fk = __uint_as_float((uint32_t)powers[k0 + 8 * y] << 23);
                        fv[y] = (float)(int)powers[C::kTokens + k0 + 8 * y] - 127.f;
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float z = (c0[b][2 * y + e] + c1[b][2 * y + e]) * qs[b][e];
                            sc[b][2 * y + e] = QZ ? z * fk : z;
                        }
                }
                if (left < k0 + 16 || bad) {
                    // tokens behind the sequence or on bad pages: no score, and their V rows (which may
                    // hold anything) become zero
                    const int nk = max(0, min(C::kTokens, left));
                    auto hidden = [&](int k) { return k >= nk || ((bad >> (k >> lb)) & 1u); };
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (hidden(k0 + 8 * y + g8))
#pragma unroll
                            for (int b = 0; b < NB; ++b) sc[b][2 * y] = sc[b][2 * y + 1] = -INFINITY;
                    for (int k = k0; k < k0 + 16; ++k)
                        if (hidden(k) && lane < C::kRowBytes / 16)
                            *reinterpret_cast<uint4*>(sm + (size_t)s * 2 * C::kHalf + C::kHalf + chunk_at(k, lane)) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();        // (before the ring's next copy lands on these rows)
                    __syncwarp();
                }
                // ---- running maximum, weights ----
                uint32_t pb[NB][2], pr[kTwo ? NB : 1][2];              // tokens 2 q4, + 1 (+ 8) of row 8 b + g8
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float top[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[e] = QZ ? fmaxf(sc[b][e] + fv[0], sc[b][2 + e] + fv[1]) : fmaxf(sc[b][e], sc[b][2 + e]);
#pragma unroll
                        for (int z = 4; z < kWarp; z <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], z));
                        top[e] += kRaise;
                    }
                    const bool need[2] = {top[0] > m[b][0] + kRaise, top[1] > m[b][1] + kRaise};
                    // (QZ: the lane's own scores)
                    const float own[2] = {fmaxf(sc[b][0], sc[b][2]), fmaxf(sc[b][1], sc[b][3])};
                    const bool more = QZ && (own[0] > ml[b][0] || own[1] > ml[b][1]);
                    if (__any_sync(0xffffffffu, need[0] || need[1] || more)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float f = need[e] ? ex2(m[b][e] - top[e]) : 1.f;
                            if (need[e]) m[b][e] = top[e];
                            if constexpr (QZ) {
                                const float now = own[e] > ml[b][e] ? own[e] + kRaise : ml[b][e];
                                l[b][e] *= ex2(ml[b][e] - now);
                                ml[b][e] = now;
                            } else {
                                l[b][e] *= f;
                            }
#pragma unroll
                            for (int y = 0; y < D / 16; ++y) {
                                o[y][b][e] *= f;
                                o[y][b][2 + e] *= f;
                            }
                        }
                    }
                    float w[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int e = z & 1;
                        if constexpr (QZ) {
                            w[z] = ex2(sc[b][z] + fv[z >> 1] + (kUpBits - m[b][e]));
                            l[b][e] += ex2(sc[b][z] - ml[b][e]);
                        } else {
                            w[z] = ex2(sc[b][z] - (m[b][e] == -INFINITY ? 0.f : m[b][e]));
                            l[b][e] += w[z];
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t h = QZ ? half2_of(w[2 * y], w[2 * y + 1]) : pack2(w[2 * y], w[2 * y + 1]);
                        pb[b][y] = turned(h);
                        if constexpr (kTwo) pr[b][y] = turned(half2_rest(w[2 * y], w[2 * y + 1], h));
                    }
                }
                // ---- O^T += V^T P^T ----
                if constexpr (QZ) {
#pragma unroll
                    for (int y = 0; y < D / 32; ++y) {
                        uint32_t vb[4];
                        ldsm4_t(vt + chunk_at(k0 + vrow, 2 * y + vch), vb);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t va[4];                            // channels 2 g8, 2 g8 + 1: tokens 2 q4, + 1; then + 8, + 9
                            widen(__byte_perm(vb[2 * z], 0u, 0x3120), va[0], va[1]);
                            widen(__byte_perm(vb[2 * z + 1], 0u, 0x3120), va[2], va[3]);
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                mma16816_h(o[2 * y + z][b], va, pb[b][0], pb[b][1]);
                                if constexpr (kTwo) mma16816_h(o[2 * y + z][b], va, pr[b][0], pr[b][1]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < D / 16; ++y) {
                        uint32_t va[4];
                        ldsm4_t(vt + chunk_at(k0 + vrow, 2 * y + vch), va);
#pragma unroll
                        for (int b = 0; b < NB; ++b) mma16816(o[y][b], va, pb[b][0], pb[b][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive1(smem_u32(&bars.empty[s]));
        }
        // ---- the group's end: its warps in order ----
        const int buf = turn & 1;
        if (groups > 1 && ok) ok = count_wait(&joined[buf], turn >> 1, &abort_sm);    // (the parts before are read)
        if (group_or<NT>(1 + grp, !ok)) {
            if (gt == 0) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
            break;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = m[b][e];
                if constexpr (QZ) {
                    top = ml[b][e];
#pragma unroll
                    for (int z = 4; z < kWarp; z <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
                    l[b][e] *= ex2(ml[b][e] - top - kRoom);
                    top = top == kNone ? -INFINITY : top + kRoom;
                }
#pragma unroll
                for (int z = 4; z < kWarp; z <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], z);
                if (g8 == 0) {
                    x.ms[grp][w4][8 * b + q2 + e] = top;
                    x.ls[grp][w4][8 * b + q2 + e] = l[b][e];
                }
            }
        bar();
        float f[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mm = -INFINITY;
#pragma unroll
                for (int w = 0; w < 4; ++w) mm = fmaxf(mm, x.ms[grp][w][8 * b + q2 + e]);
                // (QZ: 2^{m - 15 - mm}, which may be far from one, by its square root)
                const float to = m[b][e] - (mm == -INFINITY ? 0.f : mm);
                f[b][e] = QZ ? ex2(0.5f * (to - kUpBits)) : ex2(to);
            }
        float* rec = segment_record<D, SH>(a, g);
        const int er = 4 * gt / CK, ec = 4 * gt % CK;                          // 128 threads x 4 columns = 8 NB x CK
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) mm = fmaxf(mm, x.ms[grp][w][er]);
#pragma unroll
        for (int w = 0; w < 4; ++w) ll = fmaf(x.ls[grp][w][er], ex2(x.ms[grp][w][er] - (mm == -INFINITY ? 0.f : mm)), ll);
#pragma unroll
        for (int c = 0; c < D; c += CK) {
            if (c > 0) bar();
#pragma unroll
            for (int y = 0; y < CK / 16; ++y)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float(&z)[4] = o[c / 16 + y][b];
                        float* to = &x.red[grp][w4][8 * b + q2 + e][16 * y];
                        if constexpr (QZ) {
                            *reinterpret_cast<float2*>(to + 2 * g8) = make_float2(z[e] * f[b][e] * f[b][e], z[2 + e] * f[b][e] * f[b][e]);
                        } else {
                            to[g8] = z[e] * f[b][e];
                            to[8 + g8] = z[2 + e] * f[b][e];
                        }
                    }
            bar();
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 z = *reinterpret_cast<const float4*>(&x.red[grp][w][er][ec]);
                y[0] += z.x;
                y[1] += z.y;
                y[2] += z.z;
                y[3] += z.w;
            }
            if (groups > 1) store4(&x.part[buf][grp][er][c + ec], y);
            else if (er < g.R) write_out<TO, D, SH>(a, g, g.whole, rec, er, c + ec, y, mm, ll);
        }
        if (groups > 1) {
            // ---- the groups in order, by the last of them ----
            if (ec == 0) {
                x.part_ml[buf][grp][0][er] = mm;
                x.part_ml[buf][grp][1][er] = ll;
            }
            __threadfence_block();
            bar();
            if (gt == 0) go[grp] = atomicAdd(&here[buf], 1) == groups - 1;
            bar();
            if (!go[grp]) continue;
            __threadfence_block();
            for (int e = gt; e < g.R * (D / 4); e += NT) {
                const int r = e / (D / 4), c = e % (D / 4) * 4;
                float top = -INFINITY, sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
                auto has = [&](int k) { return (k + kGroups - g.n0 % kGroups) % kGroups < g.tiles; };
#pragma unroll
                for (int k = 0; k < kGroups; ++k)
                    if (has(k)) top = fmaxf(top, x.part_ml[buf][k][0][r]);
#pragma unroll
                for (int k = 0; k < kGroups; ++k) {
                    if (!has(k)) continue;
                    const float w = ex2(x.part_ml[buf][k][0][r] - (top == -INFINITY ? 0.f : top));
                    const float4 z = *reinterpret_cast<const float4*>(&x.part[buf][k][r][c]);
                    sum = fmaf(w, x.part_ml[buf][k][1][r], sum);
                    y[0] = fmaf(w, z.x, y[0]);
                    y[1] = fmaf(w, z.y, y[1]);
                    y[2] = fmaf(w, z.z, y[2]);
                    y[3] = fmaf(w, z.w, y[3]);
                }
                write_out<TO, D, SH>(a, g, g.whole, rec, r, c, y, top, sum);
            }
            bar();
            if (gt == 0) {
                here[buf] = 0;
                __threadfence_block();
                *reinterpret_cast<volatile int*>(&joined[buf]) = (turn >> 1) + 1;
            }
        }
        if (!SH && !g.whole) join_pieces<TO, D, NT>(a, g, gt, &go[grp], bars.arrived, bar);
    }
    __syncthreads();
    if (abort_sm) settle<D, C::kStages, NS, SH, M::kAll * kWarp, C::kTokens, PRE>(a, bars);
}

template <typename T, typename TO, int D, int NB, bool SH, bool PRE>
cudaError_t launch_t(const DecodeArgs& d, cudaStream_t st) {
    using M = TSmem<T, TO, D, NB>;
    using C = Ring<Cfg<T, D>, M::kRing>;
    static_assert(C::kSmem + sizeof(M) + 2048 <= 232448, "ring, joins and the barriers beside them");
    static std::atomic<uint64_t> done{0};
    return launch_kernel<T, D>(decode_t_kernel<T, TO, D, NB, SH, PRE>, M::kAll, done, d, st, C::kSmem + (int)sizeof(M));
}
// (rows of a prefix: as many as its sequences have)
template <typename T, typename TO, int D, bool SH, bool PRE = false> cudaError_t launch_t(const DecodeArgs& d, cudaStream_t st) {
    return (!SH || d.sh.each) && d.p.G <= 8 ? launch_t<T, TO, D, 1, SH, PRE>(d, st) : launch_t<T, TO, D, 2, SH, PRE>(d, st);
}
template <bool SH, bool PRE = false> cudaError_t launch_quant(const DecodeArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_t<uint8_t, float, 128, SH, PRE>(a, st) : launch_t<uint8_t, float, 64, SH, PRE>(a, st);
    return a.p.d == 128 ? launch_t<uint8_t, __nv_bfloat16, 128, SH, PRE>(a, st) : launch_t<uint8_t, __nv_bfloat16, 64, SH, PRE>(a, st);
}

// ---- the cached rows as rows ----
// Row r of the packed output is a token of the sequence whose tokens, counted from the first sequence's on, hold
// number r.  Each CTA adds the lengths up for itself, looks its rows' pages up, and has NU units of 16 bytes of
// output, of K and of V, in flight a thread.  Bound by bytes: each code read once, each number written once (16
// sequences of 1000-8001 tokens, 8 heads, d = 128, bfloat16: 57 us, 5.9 TB/s; 68 with a division a unit).
constexpr int kReadRows = 32, kReadThreads = 256;

// 16 / sizeof(T) codes (4 or 8 bytes) times f
template <typename T> struct ReadUnit;
template <> struct ReadUnit<float> {
    using Codes = uint32_t;
    static __device__ __forceinline__ uint4 of(uint32_t w, float f) {
        uint32_t lo, hi;
        widen(w, lo, hi);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        return make_uint4(__float_as_uint(x.x * f), __float_as_uint(x.y * f), __float_as_uint(y.x * f), __float_as_uint(y.y * f));
    }
};
template <> struct ReadUnit<__nv_bfloat16> {
    using Codes = uint2;
    static __device__ __forceinline__ uint4 of(uint2 w, float f) {
        const uint4 x = ReadUnit<float>::of(w.x, f), y = ReadUnit<float>::of(w.y, f);
        auto pair = [](uint32_t a, uint32_t b) { return pack2(__uint_as_float(a), __uint_as_float(b)); };
        return make_uint4(pair(x.x, x.y), pair(x.z, x.w), pair(y.x, y.y), pair(y.z, y.w));
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) quant_read_kernel(const ReadArgs a) {
    constexpr int VN = 16 / sizeof(T), UH = D / VN;                    // numbers of a unit, units of a head
    __shared__ int64_t sums[kReadThreads / kWarp];
    __shared__ int64_t from[kReadRows];                                // token, then (page, slot) of a row: -1 zeros, -2 no row
    __shared__ int seq[kReadRows];
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
            seq[r - r0] = b;
            from[r - r0] = r - lo;
        }
        before = all;
        if (blockIdx.x > 0 && before >= r1) break;
    }
    __syncthreads();
    // (a lookup a thread, of all rows at once)
    if (threadIdx.x < kReadRows && from[threadIdx.x] >= 0) {
        const int64_t pos = from[threadIdx.x];
        const int page = paged_page(p, seq[threadIdx.x], pos);
        if (page < 0) bits |= LOLA_ATTN_BAD_PAGE;
        from[threadIdx.x] = page < 0 ? -1 : (int64_t)page * p.Hkv * p.page + (pos & (p.page - 1));
    }
    if (bits) atomicOr(&g_status, bits);
    __syncthreads();
    // K and V of NU units a thread are under way at once.  Unit e is part w of row i; from unit to unit the next one is
    // found without a division.
    constexpr int NU = 4;
    const int per = p.Hkv * UH, step_i = kReadThreads / per, step_w = kReadThreads - step_i * per;
    int i = (int)threadIdx.x / per, w = (int)threadIdx.x - i * per;
    while (i < kReadRows) {
        // (loads without conditions, from the pool's first row where there is nothing to read)
        typename ReadUnit<T>::Codes c[2][NU];
        uint8_t power[2][NU];
        int row_of[NU], part_of[NU];
        uint32_t zero = 0u, none = 0u;
#pragma unroll
        for (int x = 0; x < NU; ++x) {
            const int64_t at = i < kReadRows ? from[i] : -2;
            const int64_t row = at < 0 ? 0 : at + (int64_t)(w / UH) * p.page;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                c[kv][x] = *reinterpret_cast<const typename ReadUnit<T>::Codes*>((kv ? p.V : p.K) + row * D + w % UH * VN);
                power[kv][x] = (kv ? p.Vs : p.Ks)[row];
            }
            if (at < 0) zero |= 1u << x;
            if (at == -2) none |= 1u << x;
            row_of[x] = i;
            part_of[x] = w;
            i += step_i;
            w += step_w;
            if (w >= per) {
                w -= per;
                ++i;
            }
        }
#pragma unroll
        for (int x = 0; x < NU; ++x)
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const Rows& out = kv ? a.V : a.K;
                const uint4 y = ReadUnit<T>::of(c[kv][x], __uint_as_float((uint32_t)power[kv][x] << 23));
                if (!((none >> x) & 1u))
                    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(out.data) + (r0 + row_of[x]) * out.row + (int64_t)(part_of[x] / UH) * out.head +
                                              part_of[x] % UH * VN) = (zero >> x) & 1u ? make_uint4(0, 0, 0, 0) : y;
            }
    }
}
template <typename T, int D> cudaError_t launch_read(const ReadArgs& a, cudaStream_t st) {
    const unsigned grid = a.total > 0 ? (unsigned)((a.total + (int64_t)kReadRows - 1) / kReadRows) : 1u;
    return launch_behind(quant_read_kernel<T, D>, grid, kReadThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_quant_decode(const DecodeArgs& a, cudaStream_t st) { return launch_quant<false>(a, st); }
cudaError_t launch_quant_parts(const DecodeArgs& a, cudaStream_t st) { return launch_quant<true>(a, st); }
cudaError_t launch_bf16_parts(const DecodeArgs& a, cudaStream_t st) {
    return a.p.d == 128 ? launch_t<__nv_bfloat16, __nv_bfloat16, 128, true>(a, st) : launch_t<__nv_bfloat16, __nv_bfloat16, 64, true>(a, st);
}
cudaError_t launch_tiles_behind(const DecodeArgs& a, cudaStream_t st) {
    if (a.p.Ks) return launch_quant<false, true>(a, st);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, __nv_bfloat16, 128, false, true>(a, st)
                        : launch_t<__nv_bfloat16, __nv_bfloat16, 64, false, true>(a, st);
}

cudaError_t launch_quant_read(const ReadArgs& a, cudaStream_t st) {
    if (a.p.dtype == LOLA_F32) return a.p.d == 128 ? launch_read<float, 128>(a, st) : launch_read<float, 64>(a, st);
    return a.p.d == 128 ? launch_read<__nv_bfloat16, 128>(a, st) : launch_read<__nv_bfloat16, 64>(a, st);
}

cudaError_t quant_status_word(int32_t** word) { return cudaGetSymbolAddress((void**)word, g_status); }

}  // namespace lola
