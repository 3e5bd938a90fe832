// Tree decoding: parameters and launchers of the operators that score a tree
// of drafted tokens (tree_attn.cuh, tree_attn_q8.cuh), turn logits into token probabilities,
// verify the drafts and commit the kept ones to the K/V cache (tree.cu).
// Every kernel here is stateless: work split over several CTAs is joined
// inside a thread block cluster through distributed shared memory, so no call
// needs a workspace, and calls on any streams or in any graphs share nothing.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace llmq {

// How long a device-side wait of these kernels may take. The test hook makes a
// barrier of each CTA expect a warp's arrivals more than it gets, with a short limit.
struct WaitLimit {
  uint32_t ns = 2000000000;
  int missing = 0;
};
extern std::atomic<bool> g_expire_waits;  // llm_debug_expire_waits
inline WaitLimit wait_limit() { return g_expire_waits.load(std::memory_order_relaxed) ? WaitLimit{1000000, 32} : WaitLimit{}; }

constexpr int kTreeMaxNodes = 64;  // a node's visible set is one 64-bit word

// A kernel's dynamic shared memory limit (and the leave for clusters of 16), set once per device (one of these,
// static, beside each kernel's launch: its size never changes).
class SmemLimit {
 public:
  template <typename Kern>
  cudaError_t raise(Kern kern, int bytes, bool cluster16 = false) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done_.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && cluster16) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev < 64) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// How many clusters of `size` CTAs (a power of two up to 16) the device runs at
// once, asked once per device and size.
class ClusterCount {
 public:
  template <typename Kern>
  int get(Kern kern, int size, int threads, size_t smem) {
    int dev = 0, lg = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    while ((1 << lg) < size) ++lg;
    std::atomic<int>* slot = dev < kDevices ? &n_[dev][lg] : nullptr;
    if (slot && (n = slot->load(std::memory_order_relaxed))) return n;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = n > 0 ? n : -1;
    if (slot) slot->store(n, std::memory_order_relaxed);
    return n;
  }

 private:
  static constexpr int kDevices = 16;
  std::atomic<int> n_[kDevices][5] = {};
};

// Launch in clusters along x (of one CTA: none), as a programmatic dependent:
// the launch and a kernel's set-up overlap the end of the kernel before it. Every
// kernel launched so waits (griddepcontrol) before its first access to global
// memory, in every thread, so stream order holds as without it.
template <typename Kern, typename Params>
cudaError_t launch_cluster(Kern kern, dim3 grid, int threads, int cluster, size_t smem, cudaStream_t st,
                           const Params& p, bool pdl = true) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// x / d as one multiplication, exact while x d < 2^32 (the callers check).
struct FastDiv {
  uint32_t mul = 0;
  FastDiv() = default;
  explicit FastDiv(int d) : mul(d > 1 ? (uint32_t)((0x100000000ull + d - 1) / d) : 0) {}
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int x) const { return mul ? (int)__umulhi((uint32_t)x, mul) : x; }
#endif
};

struct KvRows {              // K and V rows of one layer: a cache, or the drafted tree's own
  const uint8_t* k = nullptr;      // bf16 values, or int8 codes (then the scales are set)
  const uint8_t* v = nullptr;
  const uint16_t* ks = nullptr;    // fp16 scales of each 32 values
  const uint16_t* vs = nullptr;
  int64_t seq = 0, head = 0, row = 0;     // strides in elements of k and v
  int64_t sseq = 0, shead = 0, srow = 0;  // strides of the scales
  int rows = 0;                    // rows a head holds
};

struct TreeAttnParams {
  const void* q;             // bf16 or fp32
  void* out;                 // the type of q
  int64_t q_seq, q_node, q_head, o_seq, o_node, o_head;  // strides in elements
  KvRows cache, tree;        // tree.k null: the cache alone
  const int* lens;           // [B] cache rows that every node sees
  const uint64_t* mask;      // [B][n] tree rows that a node sees
  const int* counts;         // [B] nodes of a sequence, or null: n
  int64_t mask_seq;
  float c;                   // |scale| log2(e), above 0
  bool neg = false;          // the scale is negative: the queries change their signs
  int B, n, Hkv, gq;
  FastDiv by_gq;
  int S;                     // CTAs of a cluster: splits of the keys
  bool pdl = true;           // launch as a programmatic dependent
  bool sorted;               // blocks take the sequences longest first
  // Attention in two parts over different rows. kFirst: "sequence" b of the cache is one that the sequences
  // starts[b] .. starts[b + 1] - 1 (of all) share, whose nodes follow one another as its rows; the results go to
  // part_o, part_ml instead of out, in part_n pieces. kSecond: the results are joined with those of the first part,
  // launched just before it, where the sequence is in starts[0] .. starts[B] - 1.
  enum Part : int { kWhole, kFirst, kSecond } part = kWhole;
  const int* starts = nullptr;
  int G = 0, all = 0;        // groups, sequences
  int nodes;                 // most nodes of a block's sequence(s): n, or all n
  static constexpr int kMaxParts = 8;
  int* part_n = nullptr;     // [all][n][heads] pieces of a row: 0 .. max_parts, which is kMaxParts at most
  int max_parts = 1;
  int64_t part_rows = 0;     // all n heads
  float* part_o = nullptr;   // [max_parts][all][n][heads][head_dim] normalised
  float2* part_ml = nullptr; // [max_parts][all][n][heads] (reference, sum)
  FastDiv by_n;
  int* status;               // the device's status word (bounded waits)
  WaitLimit wait = wait_limit();
};

// f32: q and out are fp32 (else bf16); q8: int8 rows. n_sm: SMs of the device.
cudaError_t launch_tree_attn(const TreeAttnParams& p, int hd, bool f32, bool q8, int n_sm, cudaStream_t st);
cudaError_t launch_tree_attn_64(const TreeAttnParams& p, bool f32, bool q8, int n_sm, cudaStream_t st);
cudaError_t launch_tree_attn_128(const TreeAttnParams& p, bool f32, bool q8, int n_sm, cudaStream_t st);

constexpr int kProbSlice = 51200;     // floats of a row that one CTA of 16 keeps
constexpr int kProbTopSlice = 32768;  // with top_k

struct TokenProbsParams {
  const float* logits;
  float* probs;
  int64_t l_row, p_row;      // strides in elements
  int R, V;
  float c;                   // log2(e) / temperature
  int top_k;                 // 0: every token
  float top_p;
  bool pdl = true;
  int cap = 0;               // set by the launch: floats of a slice
  int* status;               // the device's status word (bounded waits)
  WaitLimit wait = wait_limit();
};
cudaError_t launch_token_probs(const TokenProbsParams& p, int n_sm, cudaStream_t st);

struct VerifyParams {
  const int *tokens, *parents;  // [B][n]
  const int* counts;            // [B] or null
  const float* u;               // [B][n]
  const float *p, *q;           // [B][n][V]; q null: the drafts are certain choices
  int64_t p_seq, p_node, q_seq, q_node;
  const int* targets;           // [B][n] greedy mode: the target's choice after each node (p null)
  int *path, *n_path, *next;
  int B, n, V;
  bool pdl = true;
};
cudaError_t launch_verify_tree(const VerifyParams& p, int n_sm, cudaStream_t st);

struct CommitParams {
  KvRows cache, tree;        // strides of one layer; layer strides below
  int64_t c_layer, c_slayer, t_layer, t_slayer;
  const int *lens, *path, *n_path;
  int* new_lens;             // may be lens itself
  // a model's own sequence (one, new_lens is lens): where *status is set nothing is committed; the
  // next token goes where the model's steps look for it
  const int *status = nullptr, *next = nullptr;
  int *tok = nullptr, *argmax = nullptr;
  int64_t path_seq;
  FastDiv by_heads;
  bool pdl = true;
  int B, L, Hkv, n, row_bytes, srow_bytes;  // bytes of a row of k or v, and of its scales (0: none)
};
cudaError_t launch_commit_tree(const CommitParams& p, cudaStream_t st);

// The device's status word of the bounded waits (llm_tree_status).
cudaError_t status_word(int dev, int** p);

// Records the calling thread's error text of a call without a model (llm_last_error(NULL)); returns code.
int op_error(int code, const char* msg) noexcept;

}  // namespace llmq
