// embedding.hip -- rows of a table by token ids, scaled, and the table's gradient by sorted tokens.
//
// Mathematics:  out[i] = scale * table[token[i]];  dtable[v] = scale * sum of dout[i] over the i
// with token[i] = v.  A token outside [0, vocab) has a row of zeros and adds to no gradient.
//
// Order of the gradient's sums: a token's positions in ascending order, cut into blocks of 64 from
// its first on; a block is a chain of additions in f32, the blocks are added in their order in f64
// (one block: its sum as it is).  It depends on a token's own positions alone.  The sort is of
// whole numbers, and no value is added by an atomic.
#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

constexpr int64_t kBlockRows = 64;          // positions a block of the gradient's sums
constexpr int64_t kChunk = 1024;            // tokens that a workgroup sorts
constexpr int64_t kChunkSortMax = 65536;    // tokens sorted by chunks; more go through the radix sort
constexpr int kGroup = 4;                   // chunks that a wave of the ranking holds in LDS
constexpr int64_t kSlab = 64;               // vectors of a row that a wave takes: one a lane

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// token i, or `none` where it lies outside the vocabulary
__device__ __forceinline__ uint32_t token_at(const void* tokens, bool wide, int64_t i,
                                             int64_t vocab, uint32_t none) {
    const int64_t t = wide ? static_cast<const int64_t*>(tokens)[i]
                           : (int64_t)static_cast<const int32_t*>(tokens)[i];
    return t >= 0 && t < vocab ? (uint32_t)t : none;
}

struct EmbedArgs {
    const void* table;
    const void* tokens;
    void* out;
    int64_t stride, n, vocab, d;
    float scale;
    bool wide;
    int lanes_log2;      // lanes of a row: a power of two up to 256
};

// A team of lanes takes R neighbouring rows, whose tokens and then whose vectors are in flight
// together.  Bound by HBM, or for a few tokens by the latency of a token and of its row: 16384 tokens x 4096
// bf16 36 us (89 MB fetched, since tokens repeat, and 134 written: 6.2 TB/s), 64 tokens 3.
template <typename T, int R>
__global__ __launch_bounds__(256) void k_embedding(EmbedArgs a) {
    const int lanes = 1 << a.lanes_log2;
    const int team = threadIdx.x >> a.lanes_log2, t = threadIdx.x & (lanes - 1);
    const int64_t per = (int64_t)(256 >> a.lanes_log2) * R;
    for (int64_t row0 = (int64_t)blockIdx.x * per + team * R; row0 < a.n;
         row0 += (int64_t)gridDim.x * per) {
        const T* src[R];
        bool known[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t none = 0xFFFFFFFFu;
            const uint32_t id = token_at(a.tokens, a.wide, row0 + r < a.n ? row0 + r : a.n - 1,
                                         a.vocab, none);
            known[r] = id != none;
            src[r] = static_cast<const T*>(a.table) + (known[r] ? (int64_t)id : 0) * a.stride;
        }
        for (int64_t c = (int64_t)kVec<T> * t; c < a.d; c += (int64_t)kVec<T> * lanes) {
            u32x4 raw[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                raw[r] = u32x4{0, 0, 0, 0};
                if (a.vocab > 0) raw[r] = load_row(src[r], c, a.d);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (row0 + r >= a.n) break;
                float v[kVec<T>];
                unpack<T>(settle<T>(raw[r], c, a.d), v);
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i) v[i] = known[r] ? v[i] * a.scale : 0.0f;
                write_vec(static_cast<T*>(a.out) + (row0 + r) * a.d + c, a.d - c, v);
            }
        }
    }
}

// ---------------------------------------------------------------- sort by chunks

typedef unsigned long long u64;

// A step of a bitonic network over the chunk: partners STEP apart, runs of SIZE.
template <int SIZE, int STEP>
__device__ __forceinline__ void exchange(u64& key, u64* s_key) {
    const int t = threadIdx.x;
    u64 other;
    if constexpr (STEP >= 64) {
        __syncthreads();
        s_key[t] = key;
        __syncthreads();
        other = s_key[t ^ STEP];
    } else {
        uint32_t lo = (uint32_t)key, hi = (uint32_t)(key >> 32);
        if constexpr (STEP == 32) {
            lo = (uint32_t)__builtin_amdgcn_ds_bpermute((t ^ 32) << 2, (int)lo);
            hi = (uint32_t)__builtin_amdgcn_ds_bpermute((t ^ 32) << 2, (int)hi);
        } else {
            lo = xor_partner<STEP>(lo);
            hi = xor_partner<STEP>(hi);
        }
        other = (u64)hi << 32 | lo;
    }
    const bool up = (t & SIZE) == 0, low = (t & STEP) == 0;
    if ((up == low) == (other < key)) key = other;
    if constexpr (STEP > 1) exchange<SIZE, STEP / 2>(key, s_key);
}

template <int SIZE>
__device__ __forceinline__ void merge_runs(u64& key, u64* s_key) {
    if constexpr (SIZE > 2) merge_runs<SIZE / 2>(key, s_key);
    exchange<SIZE, SIZE / 2>(key, s_key);
}

// Chunk of 1024 (token, position), sorted: partners within a wave by lane moves, farther ones through
// LDS.  Positions are part of the key, so equal tokens keep their order.  Behind the last token the
// chunk holds tokens larger than any.  (7 us whatever their number: 55 exchanges one after another.)
__global__ __launch_bounds__(1024) void k_sort_chunks(const void* tokens, bool wide, int64_t n,
                                                      int64_t vocab, uint32_t* tok, uint32_t* pos) {
    __shared__ u64 s_key[kChunk];
    const int t = threadIdx.x;
    const int64_t i = (int64_t)blockIdx.x * kChunk + t;
    const uint32_t id = i < n ? token_at(tokens, wide, i, vocab, (uint32_t)vocab) : 0xFFFFFFFFu;
    u64 key = (u64)id << 32 | (uint32_t)t;
    merge_runs<kChunk>(key, s_key);
    tok[i] = (uint32_t)(key >> 32);
    pos[i] = (uint32_t)(i - t) + (uint32_t)key;
}

// Place of every token among all: its place in its chunk, and the tokens before it in the others:
// up to its own number in earlier chunks, below it in later ones.  A workgroup takes 64 tokens; each of
// its waves searches every fourth group of four chunks, in LDS of its own, whose loads are all in flight
// at once (32768 tokens: 6.4 us; one wave, eight chunks at a time, 14).
__global__ __launch_bounds__(256) void k_rank_tokens(const uint32_t* tok, const uint32_t* pos,
                                                     int64_t n, uint32_t* keys, uint32_t* src) {
    constexpr int kWaves = 4, kLoads = kGroup * (int)kChunk / 256;
    __shared__ __attribute__((aligned(16))) uint32_t s_group[kWaves][kGroup * kChunk];
    __shared__ uint32_t s_before[kWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t e = (int64_t)blockIdx.x * 64 + lane;      // of the padded length
    const int chunks = (int)((n + kChunk - 1) / kChunk), own = (int)((int64_t)blockIdx.x * 64 / kChunk);
    const uint32_t id = tok[e];
    uint32_t* const s_tok = s_group[wave];
    uint32_t before = 0;
    for (int c0 = wave * kGroup; c0 < chunks; c0 += kWaves * kGroup) {
        u32x4 raw[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {      // chunks past the last one as that
            const int c = c0 + u * kGroup / kLoads < chunks ? c0 + u * kGroup / kLoads : chunks - 1;
            raw[u] = *reinterpret_cast<const u32x4*>(tok + (int64_t)c * kChunk + u % (kLoads / kGroup) * 256 +
                                                     lane * 4);
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) *reinterpret_cast<u32x4*>(s_tok + u * 256 + lane * 4) = raw[u];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint32_t at[kGroup] = {};
#pragma unroll
        for (int step = kChunk / 2; step > 0; step /= 2)
#pragma unroll
            for (int c = 0; c < kGroup; ++c) {
                const uint32_t bound = id + (c0 + c < own ? 1u : 0u);
                if (s_tok[c * kChunk + at[c] + step - 1] < bound) at[c] += step;
            }
#pragma unroll
        for (int c = 0; c < kGroup; ++c) {
            const uint32_t bound = id + (c0 + c < own ? 1u : 0u);
            if (s_tok[c * kChunk + at[c]] < bound) at[c] += 1;
            if (c0 + c < chunks && c0 + c != own) before += at[c];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    s_before[wave][lane] = before;
    __syncthreads();
    if (wave == 0 && id != 0xFFFFFFFFu) {
        const uint32_t place = (uint32_t)(e % kChunk) + s_before[0][lane] + s_before[1][lane] +
                               s_before[2][lane] + s_before[3][lane];
        keys[place] = id;
        src[place] = pos[e];
    }
}

// off[v]: the first place with a token of v or more (65536 of 32768 tokens: 5 us of dependent loads)
__global__ __launch_bounds__(256) void k_token_offsets(const uint32_t* keys, int64_t n,
                                                       int64_t vocab, uint32_t* off) {
    for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v <= vocab; v += (int64_t)gridDim.x * 256) {
        uint32_t lo = 0, hi = (uint32_t)n;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (keys[mid] < (uint32_t)v)
                lo = mid + 1;
            else
                hi = mid;
        }
        off[v] = lo;
    }
}

// the radix sort's 32-bit indices
__global__ __launch_bounds__(256) void k_narrow_tokens(const void* tokens, int64_t n, int64_t vocab,
                                                       int32_t* index) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        index[i] = (int32_t)token_at(tokens, true, i, vocab, 0xFFFFFFFFu);
}

// ---------------------------------------------------------------- gradient

struct EmbedBackArgs {
    const void* dout;
    const uint32_t *keys, *src, *off;
    float* part;          // [2 * ranges][d]: blocks of tokens with several
    void* dtable;
    int64_t stride, n, vocab, d, slabs;
    float scale;
};

// The block of a token with several that begins at place p: at most one of a range of 64 places
// is its token's first, and at most one is not.
__device__ __forceinline__ int64_t block_slot(int64_t p, bool first) {
    return 2 * (p / kBlockRows) + (first ? 1 : 0);
}

// acc += the rows at places begin .. end (at most 64), one after another: a vector a lane
template <typename T>
__device__ __forceinline__ void add_rows(const EmbedBackArgs& a, int64_t begin, int64_t end,
                                         int64_t c, float (&acc)[kVec<T>]) {
    constexpr int kAhead = 8;      // rows in flight
    const int lane = threadIdx.x & 63, count = (int)(end - begin);
    const uint32_t mine = a.src[begin + (lane < count ? lane : count - 1)];
    const T* rows = static_cast<const T*>(a.dout);
    for (int k = 0; k < count; k += kAhead) {
        u32x4 raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int at = k + u < count ? k + u : count - 1;
            const int64_t row = (uint32_t)__builtin_amdgcn_readlane((int)mine, at);
            raw[u] = u32x4{0, 0, 0, 0};
            if (c < a.d) raw[u] = load_row(rows + row * a.stride, c, a.d);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (k + u < count) {
                float v[kVec<T>];
                unpack<T>(settle<T>(raw[u], c, a.d), v);
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i) acc[i] += v[i];
            }
        }
    }
}

// The blocks that begin in a range of 64 places, of tokens with more than 64 positions: bit l of the
// result is set where one begins at place l; `first` and `end` are the places of its token.
__device__ __forceinline__ uint64_t blocks_of(const EmbedBackArgs& a, int64_t range, uint32_t& first,
                                              uint32_t& end) {
    const int64_t p = range * kBlockRows + (threadIdx.x & 63);
    bool begins = false;
    first = end = 0;
    if (p < (int64_t)a.off[a.vocab]) {
        const uint32_t v = a.keys[p];
        first = a.off[v];
        end = a.off[v + 1];
        begins = end - first > kBlockRows && ((uint32_t)p - first) % kBlockRows == 0;
    }
    return __ballot(begins);
}

// Sums of the blocks of tokens with more than 64 positions: a wave per range and slab of columns.
template <typename T>
__device__ __forceinline__ void sum_blocks(const EmbedBackArgs& a, int64_t item) {
    const int64_t range = item / a.slabs, c = (item % a.slabs * kSlab + (threadIdx.x & 63)) * kVec<T>;
    uint32_t first, end;
    for (uint64_t left = blocks_of(a, range, first, end); left; left &= left - 1) {
        const int at = __builtin_ctzll(left);
        const int64_t begin = range * kBlockRows + at;
        const int64_t start = (uint32_t)__builtin_amdgcn_readlane((int)first, at);
        const int64_t stop = (uint32_t)__builtin_amdgcn_readlane((int)end, at);
        float acc[kVec<T>] = {};
        add_rows<T>(a, begin, begin + kBlockRows < stop ? begin + kBlockRows : stop, c, acc);
        if (c < a.d)
            write_floats(a.part + block_slot(begin, begin == start) * a.d + c, a.d - c, acc);
    }
}

// A wave per kVocabRows rows of the table and slab of columns: zeros, or the sum of a token's one
// block.  The rows' positions lie side by side, so the loads run ahead across them.
constexpr int kVocabRows = 8;

template <typename T>
__device__ __forceinline__ void sum_rows(const EmbedBackArgs& a, int64_t item) {
    constexpr int kAhead = 8;      // rows of dout in flight
    const int lane = threadIdx.x & 63;
    const int64_t v0 = item / a.slabs * kVocabRows, c = (item % a.slabs * kSlab + lane) * kVec<T>;
    const int64_t bound = v0 + lane < a.vocab ? v0 + lane : a.vocab;
    const int off = (int)a.off[lane <= kVocabRows ? bound : v0];
    const auto off_of = [&](int r) { return (uint32_t)__builtin_amdgcn_readlane(off, r); };
    const int rows = a.vocab - v0 < kVocabRows ? (int)(a.vocab - v0) : kVocabRows;
    T* out = static_cast<T*>(a.dtable) + v0 * a.d + c;
    const auto put = [&](int r, float (&acc)[kVec<T>]) {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) acc[i] *= a.scale;
        if (c < a.d) write_vec(out + r * a.d, a.d - c, acc);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) acc[i] = 0.0f;
    };
    float acc[kVec<T>] = {};
    int r = 0;
    while (r < rows) {
        // the rows up to the next token of several blocks, whose row is written once they are there
        int stop = r;
        while (stop < rows && off_of(stop + 1) - off_of(stop) <= kBlockRows) ++stop;
        const uint32_t begin = off_of(r), end = off_of(stop);
        for (uint32_t p0 = begin; p0 < end; p0 += 64) {
            const uint32_t mine = a.src[p0 + lane < end ? p0 + lane : end - 1];
            const int count = end - p0 < 64 ? (int)(end - p0) : 64;
            for (int k = 0; k < count; k += kAhead) {
                u32x4 raw[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int at = k + u < count ? k + u : count - 1;
                    const int64_t row = (uint32_t)__builtin_amdgcn_readlane((int)mine, at);
                    raw[u] = u32x4{0, 0, 0, 0};
                    if (c < a.d) raw[u] = load_row(static_cast<const T*>(a.dout) + row * a.stride, c, a.d);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (k + u < count) {
                        while (p0 + k + u >= off_of(r + 1)) put(r++, acc);
                        float v[kVec<T>];
                        unpack<T>(settle<T>(raw[u], c, a.d), v);
#pragma unroll
                        for (int i = 0; i < kVec<T>; ++i) acc[i] += v[i];
                    }
                }
            }
        }
        while (r < stop) put(r++, acc);
        ++r;      // the token of several blocks
    }
}

// Both in one launch, the blocks (the longer work) first.  Bound by HBM: dout is read once, the gradient
// written once (32768 tokens x 2048 bf16 into 65536 rows 84 us, 403 MB, 4.8 TB/s; x 768 into 50257 rows 30,
// where frequent tokens' rows come one behind the other).
template <typename T>
__global__ __launch_bounds__(256) void k_embedding_sums(EmbedBackArgs a, int64_t blocks) {
    const int64_t items = blocks + (a.vocab + kVocabRows - 1) / kVocabRows * a.slabs;
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < items;
         item += (int64_t)gridDim.x * 4) {
        if (item < blocks)
            sum_blocks<T>(a, item);
        else
            sum_rows<T>(a, item - blocks);
    }
}

// The blocks of every token that has several, joined: a wave per range, that its first block begins in.
// (32768 tokens x 2048: 9 us, one block at a time 14.)
template <typename T>
__global__ __launch_bounds__(256) void k_embedding_join(EmbedBackArgs a, int64_t blocks) {
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < blocks;
         item += (int64_t)gridDim.x * 4) {
        const int64_t range = item / a.slabs, c = (item % a.slabs * kSlab + (threadIdx.x & 63)) * kVec<T>;
        uint32_t first, end;
        for (uint64_t left = blocks_of(a, range, first, end); left; left &= left - 1) {
            const int at = __builtin_ctzll(left);
            const int64_t begin = (uint32_t)__builtin_amdgcn_readlane((int)first, at);
            const int64_t stop = (uint32_t)__builtin_amdgcn_readlane((int)end, at);
            if (begin != range * kBlockRows + at || c >= a.d) continue;
            const uint32_t v = a.keys[begin];
            double sum[kVec<T>] = {};
            if (c + kVec<T> <= a.d) {
                constexpr int kAhead = 8;      // blocks in flight
                for (int64_t p0 = begin; p0 < stop; p0 += kAhead * kBlockRows) {
                    f32x4 q[kAhead][kVec<T> / 4];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {      // past the last block the first again
                        const int64_t p = p0 + u * kBlockRows < stop ? p0 + u * kBlockRows : begin;
                        const float* part = a.part + block_slot(p, p == begin) * a.d + c;
#pragma unroll
                        for (int i = 0; i < kVec<T> / 4; ++i)
                            q[u][i] = *reinterpret_cast<const f32x4_a4*>(part + 4 * i);
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        if (p0 + u * kBlockRows < stop) {
#pragma unroll
                            for (int i = 0; i < kVec<T>; ++i) sum[i] += (double)q[u][i / 4][i % 4];
                        }
                }
            } else {
                for (int64_t p = begin; p < stop; p += kBlockRows)
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i)
                        if (c + i < a.d) sum[i] += (double)a.part[block_slot(p, p == begin) * a.d + c + i];
            }
            float acc[kVec<T>];
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) acc[i] = (float)sum[i] * a.scale;
            write_vec(static_cast<T*>(a.dtable) + (int64_t)v * a.d + c, a.d - c, acc);
        }
    }
}

// ---------------------------------------------------------------- launches

constexpr int64_t kGridMax = 1 << 21;      // workgroups a launch starts at most

template <typename T>
void embed_typed(const EmbedArgs& a, hipStream_t s) {
    const int64_t teams = 256 >> a.lanes_log2;
    KernelTimer kt("k_embedding", s);
    // four rows a team once that leaves every compute unit eight workgroups
    if (a.n >= 4 * teams * 2048) {
        int64_t g = cdiv(a.n, 4 * teams);
        if (g > kGridMax) g = kGridMax;
        k_embedding<T, 4><<<dim3((unsigned)g), dim3(256), 0, s>>>(a);
    } else {
        int64_t g = cdiv(a.n, teams);
        if (g > kGridMax) g = kGridMax;
        k_embedding<T, 1><<<dim3((unsigned)g), dim3(256), 0, s>>>(a);
    }
}

template <typename T>
det_status embed_back_typed(EmbedBackArgs a, hipStream_t s) {
    a.slabs = cdiv(a.d, kSlab * kVec<T>);
    // up to 64 positions no token has several blocks
    const int64_t blocks = a.n > kBlockRows ? cdiv(a.n, kBlockRows) * a.slabs : 0;
    const auto grid = [](int64_t waves) {
        const int64_t g = cdiv(waves, 4);
        return dim3((unsigned)(g < kGridMax ? g : kGridMax));
    };
    {
        KernelTimer kt("k_embedding_sums", s);
        k_embedding_sums<T><<<grid(blocks + cdiv(a.vocab, kVocabRows) * a.slabs), dim3(256), 0, s>>>(a, blocks);
    }
    if (blocks > 0) {
        KernelTimer kt("k_embedding_join", s);
        k_embedding_join<T><<<grid(blocks), dim3(256), 0, s>>>(a, blocks);
    }
    return launch_status();
}

struct EmbedLayout {
    size_t tok, pos, keys, src, off, index, sort, part, total;
};

EmbedLayout embed_layout(int64_t n, int64_t vocab, int64_t d) {
    EmbedLayout L = {};
    size_t o = 0;
    const auto take = [&](size_t bytes) {
        const size_t at = o;
        o += round_up(bytes > 0 ? bytes : 1, 256);
        return at;
    };
    if (n <= kChunkSortMax) {
        const size_t padded = (size_t)cdiv(n, kChunk) * kChunk * 4;
        L.tok = take(padded);
        L.pos = take(padded);
        L.keys = take((size_t)n * 4);
        L.src = take((size_t)n * 4);
        L.off = take((size_t)(vocab + 1) * 4);
    } else {
        L.index = take((size_t)n * 4);
        L.sort = take(sort_rows_workspace(n, vocab));
    }
    if (n > kBlockRows) L.part = take((size_t)(2 * cdiv(n, kBlockRows)) * d * 4);
    L.total = o;
    return L;
}

}  // namespace

size_t embedding_backward_workspace(int64_t n, int64_t vocab, int64_t d) {
    return embed_layout(n, vocab, d).total;
}

det_status embedding_launch(const EmbedCall& c, hipStream_t s) {
    EmbedArgs a{c.table, c.tokens, c.out, c.table_stride, c.n, c.vocab, c.d, c.scale, c.wide, 0};
    const int64_t vectors = cdiv(c.d, 16 / (int64_t)lm_size(c.dtype));
    while (a.lanes_log2 < 8 && (int64_t)1 << a.lanes_log2 < vectors) ++a.lanes_log2;
    switch (c.dtype) {
        case DET_F32: embed_typed<float>(a, s); break;
        case DET_F16: embed_typed<_Float16>(a, s); break;
        default: embed_typed<__bf16>(a, s); break;
    }
    return launch_status();
}

det_status embedding_backward_launch(const EmbedBackCall& c, void* ws, hipStream_t s) {
    const EmbedLayout L = embed_layout(c.n, c.vocab, c.d);
    char* w = static_cast<char*>(ws);
    EmbedBackArgs a{c.dout, nullptr, nullptr, nullptr, reinterpret_cast<float*>(w + L.part),
                    c.dtable, c.stride, c.n, c.vocab, c.d, 0, c.scale};
    if (c.n <= kChunkSortMax) {
        uint32_t* tok = reinterpret_cast<uint32_t*>(w + L.tok);
        uint32_t* pos = reinterpret_cast<uint32_t*>(w + L.pos);
        uint32_t* keys = reinterpret_cast<uint32_t*>(w + L.keys);
        uint32_t* src = reinterpret_cast<uint32_t*>(w + L.src);
        uint32_t* off = reinterpret_cast<uint32_t*>(w + L.off);
        const int64_t chunks = cdiv(c.n, kChunk);
        if (chunks > 0) {
            {
                KernelTimer kt("k_sort_chunks", s);
                k_sort_chunks<<<dim3((unsigned)chunks), dim3(kChunk), 0, s>>>(c.tokens, c.wide, c.n,
                                                                             c.vocab, tok, pos);
            }
        }
        if (chunks > 1) {
            KernelTimer kt("k_rank_tokens", s);
            k_rank_tokens<<<dim3((unsigned)(chunks * kChunk / 64)), dim3(256), 0, s>>>(
                tok, pos, c.n, keys, src);
        } else {      // in order already
            keys = tok;
            src = pos;
        }
        int64_t g = cdiv(c.vocab + 1, 256);
        if (g > kGridMax) g = kGridMax;
        KernelTimer kt("k_token_offsets", s);
        k_token_offsets<<<dim3((unsigned)g), dim3(256), 0, s>>>(keys, c.n, c.vocab, off);
        a.keys = keys;
        a.src = src;
        a.off = off;
    } else {
        const int32_t* index = static_cast<const int32_t*>(c.tokens);
        if (c.wide) {
            int32_t* narrow = reinterpret_cast<int32_t*>(w + L.index);
            int64_t g = cdiv(c.n, 256);
            if (g > 16384) g = 16384;
            KernelTimer kt("k_narrow_tokens", s);
            k_narrow_tokens<<<dim3((unsigned)g), dim3(256), 0, s>>>(c.tokens, c.n, c.vocab, narrow);
            index = narrow;
        }
        SortedRows sorted;
        const det_status st = sort_rows_launch(index, c.n, c.vocab, w + L.sort, &sorted, s);
        if (st != DET_SUCCESS) return st;
        a.keys = sorted.keys;
        a.src = sorted.src;
        a.off = sorted.off;
    }
    const det_status st = launch_status();
    if (st != DET_SUCCESS) return st;
    switch (c.dtype) {
        case DET_F32: return embed_back_typed<float>(a, s);
        case DET_F16: return embed_back_typed<_Float16>(a, s);
        default: return embed_back_typed<__bf16>(a, s);
    }
}

}  // namespace det
