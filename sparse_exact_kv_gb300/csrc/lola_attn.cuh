// Shared by the exact-attention kernels: argument blocks, the packed sequences' and the paged
// cache's index arithmetic, and the launchers.
#pragma once

#include <atomic>

#include "lola_internal.cuh"

namespace lola {

constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr float kAttnLn2 = 0.6931471805599453f;

struct Rows {
    char* data;
    int64_t row, head;   // elements
};

// a paged cache
struct PagedArgs {
    char* K;
    char* V;
    int n_pages, page, page_log2, n_seq, width;
    int64_t table_stride;
    const int32_t* table;
    const int32_t* kv_len;
    int Hq, Hkv, G, d, dtype;
    uint8_t* Ks;         // a quantised cache's powers of two [n_pages, Hkv, page] (K and V are e4m3 numbers then),
    uint8_t* Vs;         // or null
};

// Parts of softmaxes, left for a kernel that joins them (lola_shared.cu): of row (sequence, query head) i, largest score m in
// log2 units, sum l and output z against m.  One part in whole[i], ml[i], or the parts of several pieces in records, the first
// of them number desc[i].y, the others in the first of two of every desc[i].w-th CTA from there on, row desc[i].z; desc[i].x
// says how many.  Nothing is there for a row without tokens.
struct Parts {
    int4* desc;
    float* whole;          // [n_seq * Hq][d]
    float2* ml;
    float* rec;            // records of `rows` rows: z, where row r's columns 4 x .. 4 x + 3 are at r row_step + x chunk_step,
    int rows, row_step, chunk_step;      // then m [rows], l [rows]
};
__host__ __device__ constexpr int64_t part_record(int rows, int d) { return (int64_t)rows * (d + 2); }

// Which sequences see the tokens of entry g of a page table: g itself (each), or cu[g] .. cu[g + 1] - 1 (all, where cu is null).
struct Sharing {
    const int32_t* cu;
    int n_seq, each;
};

// one lola_attn_prefill or lola_paged_prefill
struct AttnArgs {
    int n_seq, total_q, total_k, Hq, G, dtype, d;
    const int32_t* cu_q;
    const int32_t* cu_k;
    Rows Q, K, V, O;
    float* lse;          // [Hq][total_q] or null
    float scale_log2;    // c log2(e): scores are kept in log2 units
    PagedArgs p;         // lola_paged_prefill: the keys and values (p.table null otherwise)
    int give_up;         // lola_selftest_attn_wait: a pair of key blocks at which every third CTA gives up
};

// ---- packed sequences ----
// Rows [begin, begin + len) of sequence b; malformed offsets make it empty (and set a bit of *bits).
__host__ __device__ inline void seq_rows(const int32_t* cu, int b, int total, int* begin, int* len, int* bits) {
    const int lo = cu[b], hi = cu[b + 1];
    if (lo < 0 || hi < lo || hi > total) {
        *bits |= LOLA_ATTN_BAD_OFFSETS;
        *begin = 0;
        *len = 0;
        return;
    }
    *begin = lo;
    *len = hi - lo;
}

// ---- the paged cache ----
__host__ __device__ inline int64_t paged_tokens(const PagedArgs& p, int len) {
    const int64_t most = (int64_t)p.width << p.page_log2;
    return len <= 0 ? 0 : (len > most ? most : len);
}
// the page of token pos of sequence b (pos < width * page), or -1 where it is not in the pool
__host__ __device__ inline int paged_page(const PagedArgs& p, int b, int64_t pos) {
    const int e = p.table[(int64_t)b * p.table_stride + (pos >> p.page_log2)];
    return e >= 0 && e < p.n_pages ? e : -1;
}
__host__ __device__ inline int64_t paged_offset(const PagedArgs& p, int page, int head, int64_t pos) {
    return (((int64_t)page * p.Hkv + head) * p.page + (pos & (p.page - 1))) * p.d;
}

// The keys of sequence b: packed rows [begin, begin + len), or its tokens in the cache (PG; begin = 0).
template <bool PG>
__device__ __forceinline__ void seq_keys(const AttnArgs& a, int b, int* begin, int* len, int* bits) {
    if constexpr (PG) {
        const int n = a.p.kv_len[b];
        *begin = 0;
        *len = (int)paged_tokens(a.p, n);
        if (n > *len && n > 0) *bits |= LOLA_ATTN_BAD_PAGE;
    } else {
        seq_rows(a.cu_k, b, a.total_k, begin, len, bits);
    }
}

// The sequence that row t belongs to, one warp: the last b with cu[b] <= t, found 32 offsets at a time; -1 if none.
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
// Piece c of n equal pieces of `total` units: [split_at(c), split_at(c + 1)).  (Divisions of 64 bits take hundreds of
// clocks, and a kernel begins with half a dozen of them: 32 bits where they do.)
__host__ __device__ inline int64_t split_at(int64_t total, int n, int c) {
    const int64_t x = total * c;
    return x >> 32 ? x / n : (int64_t)((uint32_t)x / (uint32_t)n);
}
__host__ __device__ inline int divide(int64_t x, int by, int* rest) {
    const int q = x >> 32 ? (int)(x / by) : (int)((uint32_t)x / (uint32_t)by);
    *rest = (int)(x - (int64_t)q * by);
    return q;
}
// the piece that holds unit u < total
__host__ __device__ inline int split_of(int64_t total, int n, int64_t u) {
    const int64_t x = u * n;
    int c = (x | total) >> 32 ? (int)(x / total) : (int)((uint32_t)x / (uint32_t)total);
    while (c + 1 < n && split_at(total, n, c + 1) <= u) ++c;
    while (c > 0 && split_at(total, n, c) > u) --c;
    return c;
}

// ---- block-wide sums over sequences (NT threads, all of them) ----
template <int NT, typename I>
__device__ __forceinline__ I block_total(I x, I* sm) {
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (lane == 0) sm[warp] = x;
    __syncthreads();
    I t = 0;
#pragma unroll
    for (int w = 0; w < NT / kWarp; ++w) t += sm[w];
    return t;
}
// Tile u of the packed queries (NT threads, all of them): the sequences' tiles of `rows` query rows are
// counted in order and taken backwards, so that the CTAs that start last have the first sequence's first
// (shortest) tiles.  False if there is no such tile.  Each thread looks at one sequence of up to NT, all
// four of its offsets at once: one round of loads, then a scan.
struct TilePos {
    int b, q0, lq, k0, lk, tile;
    int bits;            // what is wrong with offsets or lengths (thread-local: what this thread has seen)
};
template <int NT, int rows, bool PG>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int u, TilePos* pos) {
    __shared__ int sums[NT / kWarp];
    __shared__ TilePos found;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    TilePos own;
    pos->bits = 0;
    auto look = [&](int b) -> int {
        own.b = b;
        own.q0 = own.lq = own.k0 = own.lk = 0;
        if (b >= a.n_seq) return 0;
        seq_rows(a.cu_q, b, a.total_q, &own.q0, &own.lq, &pos->bits);
        seq_keys<PG>(a, b, &own.k0, &own.lk, &pos->bits);
        return (own.lq + rows - 1) / rows;
    };
    int n = 0;
    for (int b = threadIdx.x + NT; b < a.n_seq; b += NT) n += look(b);
    const int n0 = look(threadIdx.x);
    const int total = block_total<NT>(n + n0, sums);
    if (u >= total) return false;
    const int want = total - 1 - u;
    int before = 0;
    for (int base = 0; base < a.n_seq; base += NT) {
        const int x = base == 0 ? n0 : look(base + threadIdx.x);
        int inc = x;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == kWarp - 1) sums[warp] = inc;
        __syncthreads();
        int pre = before, all = before;
#pragma unroll
        for (int w = 0; w < NT / kWarp; ++w) {
            if (w < warp) pre += sums[w];
            all += sums[w];
        }
        const int lo = pre + inc - x;
        if (want >= lo && want < lo + x) {
            found = own;
            found.tile = want - lo;
        }
        if (want < all) break;
        before = all;
    }
    __syncthreads();
    const int bits = pos->bits;
    *pos = found;
    pos->bits = bits;
    return true;
}

// lola_selftest_attn_wait: whether this CTA is one that gives up at block `at`, and that is one of the n from `first` on.
__device__ __forceinline__ bool gives_up(int at, int first, int n) {
    return at >= first && at - first < n && blockIdx.x % 3 == (unsigned)at % 3;
}

// Opts a kernel in to `bytes` of dynamic shared memory, once per device (`done`: the kernel's own,
// one bit per device; the call costs about a microsecond).
template <typename K>
cudaError_t opt_in_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// These kernels are launched behind the stream's last kernel without waiting for its end: a CTA may start when
// that one's CTAs are done (or let it), sets up its barriers, and waits here before it touches global memory
// -- every CTA, so that a kernel that is done says that all before it are.  In a stream, one sequence of 1000
// tokens 12.2 -> 9.1 us a call, five short prompts 12.3 -> 9.9.  (They do not let the next kernel start before
// their end: its first, longest CTAs would gather on the SMs that are free first; float32 prompts 63 -> 68 us.)
__device__ __forceinline__ void wait_for_last_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- launchers ----
cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st);       // bf16 (lola_attn_tc.cu)
struct AppendArgs {
    PagedArgs p;
    int n_tokens, rot, pairs;
    const int32_t* cu_new;
    Rows K, V, Q, QO;        // Q.data null: keys and values only
    const float* inv_freq;
    const int32_t* positions;
};
cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t st);
int64_t paged_decode_workspace(int d);
struct DecodeArgs {
    PagedArgs p;             // launch_*_parts: of the prefixes, or of the sequences' own tokens
    PagedArgs pre;           // launch_*_behind: the prefixes (sh says whose)
    Sharing sh;
    Parts parts;             // launch_*_parts: what they leave
    Rows Q, O;
    float* lse;
    float* part;             // workspace
    uint64_t tag;            // 56 bits that no other call has
    int give_up;             // lola_selftest_attn_wait
    float scale_log2;
};
cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_f32_parts(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_bf16_parts(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_quant_parts(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_f32_behind(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_tiles_behind(const DecodeArgs& a, cudaStream_t st);      // bfloat16 and quantised caches
constexpr int kFewPrefixes = 8;                                            // ... for that many prefixes at most
constexpr int kPrefixRows = 256;         // rows of a record of launch_prefix_tc, column chunks one behind the other
cudaError_t launch_prefix_tc(const DecodeArgs& a, cudaStream_t st);       // bf16 io: prefixes
struct SharedArgs {
    PagedArgs p, prefix;     // the sequences' own tokens; the prefixes
    const int32_t* cu;
    Rows Q, O;
    float* lse;
    char* workspace;
    int give_up;
    float scale_log2;
};
int64_t shared_workspace(int n_seq, int Hq, int d, int dtype);
cudaError_t launch_shared_prefix(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_shared_own(const SharedArgs& a, cudaStream_t st);
cudaError_t launch_quant_decode(const DecodeArgs& a, cudaStream_t st);
struct ReadArgs {
    PagedArgs p;
    int total;               // rows
    Rows K, V;
    int32_t* cu;             // [n_seq + 1], written
};
cudaError_t launch_quant_read(const ReadArgs& a, cudaStream_t st);
// the address of a translation unit's anomaly word on the current device
cudaError_t attn_status_word(int32_t** word);
cudaError_t attn_tc_status_word(int32_t** word);
cudaError_t append_status_word(int32_t** word);
cudaError_t paged_status_word(int32_t** word);
cudaError_t quant_status_word(int32_t** word);
cudaError_t prefix_status_word(int32_t** word);

}  // namespace lola
