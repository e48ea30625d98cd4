// det_internal.h -- host-side declarations shared by the library's translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "det.h"

namespace det {

// Launch overrides for the shape-invariance tests (0 = default).
struct LaunchOverride {
    int grid_wgs;        // workgroups of the sum and look-back scan kernels
    int extra_lds;       // dynamic LDS bytes added to k_scan, k_sum_chunks and the radix kernels
    int sum_chunk_log2;
    int scan_A;          // test-only scan anchor constants (0 = the spec's)
    int scan_A2;
    uint32_t delay_seed; // test-only: seeded delays before the scan's status publications
    uint32_t delay_us;   //   (at most this many microseconds each; 0 = none)
};
const LaunchOverride& launch_override();
constexpr int kMaxExtraLds = 65536;   // largest extra_lds the test hook accepts

// What the most recent launches used (for the tests that show the launch shape changed).
void note_sum_grid(int64_t grid);
void note_scan_grid(int64_t grid, int64_t per_cu);

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline size_t dtype_size(det_dtype d) { return d == DET_F64 ? 8 : 4; }   // f32, i32: 4

// ---- sum
size_t sum_workspace(int64_t n, det_dtype dt);
det_status sum_launch(const void* x, int64_t n, det_dtype dt, void* out, void* ws, size_t ws_bytes,
                      hipStream_t s);
// det_sum with the partials in the library's own per-GPU array (no workspace argument)
constexpr size_t kSumNoAllocBytes = ((size_t)1 << 20) + ((size_t)1 << 14) + 256;
constexpr int kMaxDevices = 64;
det_status sum_noalloc_launch(const void* x, int64_t n, det_dtype dt, void* out, hipStream_t s);

// ---- scan
constexpr int kScanV = 32;       // elements per lane
constexpr int kScanW = 64;       // lanes per wave
constexpr int kScanWaves = 4;    // waves per tile
constexpr int kScanL = kScanW * kScanWaves;   // lanes per tile
constexpr int kScanT = kScanV * kScanL;       // elements per tile
constexpr int kScanA = 256;      // tiles per anchor interval
constexpr int kScanA2 = 256;     // anchor intervals per super-interval

size_t scan_workspace(int64_t n, det_dtype dt, unsigned flags, int64_t num_segments);
det_status scan_error(const void* ws, int32_t* out, hipStream_t s);
det_status scan_launch(const void* x, void* y, int64_t n, det_dtype dt, unsigned flags,
                       const int64_t* offs, int64_t nseg, void* ws, size_t ws_bytes,
                       hipStream_t s);

// ncols scans of n elements each (column c: x + c * n -> y + c * n) sharing flags and offsets,
// with the bits of ncols separate scan_launch calls; ws: the workspace of one n-element scan;
// cagg: scan_columns_agg_bytes(n, ncols) more bytes (tile totals of every column), 256-aligned.
det_status scan_columns_launch(const void* x, void* y, int64_t n, int64_t ncols, det_dtype dt,
                               unsigned flags, const int64_t* offs, int64_t nseg, void* ws,
                               void* cagg, hipStream_t s);
size_t scan_columns_agg_bytes(int64_t n, int64_t ncols);

// ---- scatter-add
size_t scatter_workspace(int64_t n, int64_t num_out, int64_t row_len, det_dtype dt);
// negate: every value enters negated (scatter-subtract)
det_status scatter_launch(const void* values, const int32_t* index, int64_t n, int64_t row_len,
                          det_dtype dt, void* out, int64_t num_out, void* prev, int64_t* n_skipped,
                          void* ws, size_t ws_bytes, bool negate, hipStream_t s);

// scatter-add whose prev is the running value (prev required; arguments checked by the caller)
size_t scatter_running_workspace(int64_t n, int64_t num_out, int64_t row_len, det_dtype dt);
det_status scatter_running_launch(const void* values, const int32_t* index, int64_t n,
                                  int64_t row_len, det_dtype dt, void* out, int64_t num_out,
                                  void* prev, int64_t* n_skipped, void* ws, hipStream_t s);

// Stable sort of n row indices by destination (entries outside [0, num_out) left out): keys and
// source rows in ascending (key, source) order, off[b] the first position with key >= b.
struct SortedRows {
    const uint32_t *keys, *src, *off;
};
size_t sort_rows_workspace(int64_t n, int64_t num_out);
det_status sort_rows_launch(const int32_t* index, int64_t n, int64_t num_out, void* ws,
                            SortedRows* out, hipStream_t s);

// ---- language-model operators (arguments checked by the caller)
// Inputs from this many bytes on are loaded past the caches.  Half of the 256 MB last-level cache:
// below it the producer's data may still be there, above it the loads only push out what the
// call writes.  Measured with inputs that change from call to call, plain and past the caches:
// norm of 8192 x 8192 bf16 with residual (268 MB read) 97 and 85 us, its backward over 16384 x
// 4096 111 and 99, log probabilities of 2048 x 131072 105 and 98; but norm of 2048 x 4096
// (34 MB) 12.4 and 14.5, logits' gradient of 1024 x 16384 (34 MB) 12.9 and 16.6.
constexpr size_t kOnceBytes = (size_t)128 << 20;

inline size_t lm_size(det_dtype d) { return d == DET_F32 ? 4 : d == DET_E4M3 ? 1 : 2; }

struct NormCall {
    const void *x, *residual, *weight;
    void *h, *y;
    float *scales, *rstd;
    int64_t x_stride, residual_stride, rows, d, group;
    float eps;
    det_dtype dtype;
    bool codes;        // y holds e4m3 codes
};
det_status norm_launch(const NormCall& c, hipStream_t s);

struct NormBackCall {
    const void *dy, *h, *weight, *dh;
    const float* rstd;
    void *dx, *dweight;
    int64_t dy_stride, h_stride, dh_stride, rows, d;
    det_dtype dtype;
};
size_t norm_backward_workspace(int64_t rows, int64_t d, det_dtype dtype);
det_status norm_backward_launch(const NormBackCall& c, void* ws, hipStream_t s);

struct LayerCall {
    const void *x, *residual, *weight, *bias;
    void *h, *y;
    float *mean, *rstd;
    int64_t x_stride, residual_stride, rows, d;
    float eps;
    det_dtype dtype;
};
det_status layer_norm_launch(const LayerCall& c, hipStream_t s);

struct LayerBackCall {
    const void *dy, *h, *weight, *dh;
    const float *mean, *rstd;
    void *dx, *dweight, *dbias;      // dbias NULL: not wanted
    int64_t dy_stride, h_stride, dh_stride, rows, d;
    det_dtype dtype;
};
size_t layer_norm_backward_workspace(int64_t rows, int64_t d, det_dtype dtype);
det_status layer_norm_backward_launch(const LayerBackCall& c, void* ws, hipStream_t s);

struct EmbedCall {
    const void *table, *tokens;
    void* out;
    int64_t table_stride, n, vocab, d;
    float scale;
    bool wide;         // tokens are int64, else int32
    det_dtype dtype;
};
det_status embedding_launch(const EmbedCall& c, hipStream_t s);

struct EmbedBackCall {
    const void *dout, *tokens;
    void* dtable;
    int64_t stride, n, vocab, d;
    float scale;
    bool wide;
    det_dtype dtype;
};
size_t embedding_backward_workspace(int64_t n, int64_t vocab, int64_t d);
det_status embedding_backward_launch(const EmbedBackCall& c, void* ws, hipStream_t s);

// h[t] = a[t] h[t-1] + b[t] over [batch][steps][d]
struct ScanCall {
    const void *gate, *x;
    const float* state0;       // NULL: zeros
    const int32_t* lengths;    // NULL: every sequence has all steps
    void* h;
    float* state;
    int64_t batch, steps, d;
    bool sigmoid;
    det_dtype dtype;
};
size_t gated_scan_workspace(int64_t batch, int64_t steps, int64_t d, det_dtype dtype);
det_status gated_scan_launch(const ScanCall& c, void* ws, hipStream_t s);

struct ScanBackCall {
    const void *dh, *gate, *x, *h;
    const float *state0, *dstate;      // NULL: zeros
    const int32_t* lengths;
    void *dgate, *dx;
    float* dstate0;                    // NULL: not wanted
    int64_t batch, steps, d;
    bool sigmoid;
    det_dtype dtype;
};
size_t gated_scan_backward_workspace(int64_t batch, int64_t steps, int64_t d, det_dtype dtype);
det_status gated_scan_backward_launch(const ScanBackCall& c, void* ws, hipStream_t s);

// cross entropy of softmax(scale * x weight^T)
struct XentCall {
    const void *x, *weight;
    const int64_t* targets;
    float *loss, *lse;
    int64_t x_stride, w_stride, rows, vocab, d;
    float scale;
    det_dtype dtype;
};
size_t xent_workspace(int64_t rows, int64_t vocab, int64_t d, det_dtype dtype);
det_status xent_launch(const XentCall& c, void* ws, hipStream_t s);

struct XentBackCall {
    const void *x, *weight;
    const int64_t* targets;
    const float *lse, *dloss;
    void *dx, *dweight;
    int64_t x_stride, w_stride, rows, vocab, d;
    float scale;
    det_dtype dtype;
};
size_t xent_backward_workspace(int64_t rows, int64_t vocab, int64_t d, det_dtype dtype);
det_status xent_backward_launch(const XentBackCall& c, void* ws, hipStream_t s);

constexpr int kBiasMaxSide = 128;      // buckets of one side of the relative position bias
struct BiasCall {
    const void *table, *scores;        // table NULL: the scores alone, masked
    void* out;
    int64_t sb, sh, sq;                // strides of scores (backward: of dout)
    int64_t batch, heads, q, k, q_offset, max_distance;
    const int32_t *q_offsets, *lengths;
    int buckets;
    bool bidirectional, causal;
    float fill;                        // what a masked place of out gets
    det_dtype dtype;
};
// first distance of each of a side's n buckets
void relbias_starts(int n, int64_t distance, int* starts);
det_status bias_launch(const BiasCall& c, hipStream_t s);
size_t bias_backward_workspace(int64_t batch, int64_t heads, int64_t q, int64_t k, int buckets,
                               det_dtype dtype);
det_status bias_backward_launch(const BiasCall& c, const void* dout, void* dtable, void* ws,
                                hipStream_t s);

struct LogpCall {
    const void* logits;
    const int64_t* targets;
    float *logp, *entropy, *lse, *top_logp;
    int64_t* top_ids;
    int64_t stride, rows, vocab;
    int top;
    float scale;
    det_dtype dtype;
};
det_status logprob_launch(const LogpCall& c, hipStream_t s);

struct LogpBackCall {
    const void* logits;
    const int64_t* targets;
    const float *lse, *dlogp, *entropy, *dentropy;
    void* dlogits;
    int64_t stride, dstride, rows, vocab;
    float scale;
    det_dtype dtype;
};
det_status logprob_backward_launch(const LogpBackCall& c, hipStream_t s);

// Workgroups of `block` threads of kernel `fn` with `dyn_lds` bytes of dynamic LDS that are
// resident on the current device at once (occupancy x compute units), cached per device,
// kernel and LDS size; 0 if the runtime cannot tell.  *per_cu (optional) receives the
// occupancy per compute unit.
int64_t resident_wgs(const void* fn, int block, int dyn_lds = 0, int* per_cu = nullptr);

// Compute units of the current device (cached per device); 0 if the runtime cannot tell.
int cu_count();

// Kernel timing (a test hook): while it is switched on, a KernelTimer brackets one launch with
// two HIP events on the launch's stream; det_debug_kernel_report reads them.  Off, it costs one
// relaxed load.
class KernelTimer {
  public:
    KernelTimer(const char* name, hipStream_t s);
    ~KernelTimer();
    KernelTimer(const KernelTimer&) = delete;
    KernelTimer& operator=(const KernelTimer&) = delete;

  private:
    hipStream_t s_;
    long slot_;
    unsigned gen_;
};

inline det_status launch_status() {
    return hipGetLastError() == hipSuccess ? DET_SUCCESS : DET_ERROR_LAUNCH;
}

}  // namespace det
