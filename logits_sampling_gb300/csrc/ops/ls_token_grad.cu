// ls_token_grad.cu -- loss and gradient from one call (ls_policy_loss_grad): each
// row is read once from memory, and a second time from L2.
//
// A row belongs to a CTA, or to a cluster of them.  Pass 1 adds the row up, the
// last stages of it staying in shared memory; the row's scalars follow; pass 2
// goes back from the row's end and writes the gradient.
#include "ls_token_ops.cuh"

namespace lsg {
namespace ops {

// Bound by DRAM and by what does not overlap on an SM with two rows: 2048 x 128256
// bf16 181 us (5.8 TB/s on one read and one write; 15 % of the second reads miss L2,
// which makes 6.2), 1024 x 262144 fp32 with entropies 397 (5.4 TB/s; 18 % miss L2, and
// the exchange of a row's CTAs and its scalars, barrier and membar, are a quarter of the
// stalls of its eight CTAs of 256 threads). The two calls take 232 and 461.
template <typename TIn, bool kEntropy, int T>
__global__ void __launch_bounds__(T, 1024 / T) token_grad_kernel(const TokenArgs a, int upc, int keep) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  extern __shared__ uint4 dyn_smem[];
  __shared__ Moments red[T / 32];
  __shared__ Part parts[kMaxCluster];
  __shared__ RowGradient g;
  const int tid = threadIdx.x;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t i = blockIdx.x / (unsigned)C;
  wait_for_previous();
  Run<TIn, T> run;
  run.init(a.logits, i, a.row_stride, a.vocab, upc, rank);
  Stages<TIn, T> st;
  st.init(run);
  typename Run<TIn, T>::Stage first;
  if (st.whole > 0) st.template load<LOAD_KEEP>(0, first);
  Raw* const grad = static_cast<Raw*>(a.out_grad) + i * a.grad_stride;
  RowInputs in;
  if (!counts(a, i, in.id, in.w)) {
    const bool same = run.aligned_with(grad);
    uint32_t z[8] = {};
    for (int u = tid; u < run.n; u += T) run.store(grad, same, u, z);
    if (tid == 0 && rank == 0) skip_row(a, i);
    return;  // every CTA of the row leaves here, before any cluster barrier
  }
  if (C > 1) cluster_arrive();  // the peers' shared memory may be written once all have arrived
  load_inputs<TIn>(a, i, in);
  const Kept<T> kept{dyn_smem + tid, keep};
  const float c = a.c;
  Moments r;
  bool careful = false;
#pragma unroll 1
  for (;;) {
    RowSum<kEntropy> acc;
    sum_run<LOAD_KEEP, true>(run, st, first, acc, c, careful, kept);
    r = block_moments<T / 32, kEntropy>(acc.moments(), c, red);
    if (careful || sum_ok(r)) break;  // the same in every thread
    careful = true;
    __syncthreads();  // red is read
  }
  let_next_start();
  // from the run's end: what was read last is the likeliest to be in L2
  if (st.whole > keep) st.template load<LOAD_PLAIN>(st.whole - 1 - keep, first);
  if (C > 1) cluster_moments<kEntropy>(r, careful, c, parts, C, rank);
  if (tid == 0) {
    const TokenStats s = finish_row<kEntropy, KIND_POLICY>(a, i, r, in, careful, rank == 0);
    g.init(s, s.g_lp, s.g_H, c);
  }
  __syncthreads();
  gradient_run<true>(run, st, first, g, grad, kept);
  const int place = run.place(in.id);  // the thread that has written it writes it again
  if (place >= 0 && tid == st.owner(run, place)) grad[in.id] = E::put(g.at_id);
}

// How a batch is laid out on the SMs, which hold 1024 threads of these kernels
// each.  Measured, us (threads of a CTA x CTAs of a row):
//   few rows: a row over as many CTAs as find room at once.  64 rows of 256 KB
//     256x8 11.5, 256x4 11.7, 512x2 11.8, 512x1 14.9; 8 of them 6.1, 7.2, 9.1, 11.8.
//     Rows of 64 KB: 64 of them 256x4 5.7, 512x1 6.0, 256x2 6.3, 256x8 6.8; 128 of
//     them 512x1 7.4, 256x2 8.2, 256x4 8.3; of 32 KB 64 of them 512x1 4.8, 256x2 5.4
//   more: one CTA per row, 512 threads so that fewer rows share L2 between their two
//     reads, 256 where rows are short and many.  304 rows of 256 KB 512x1 30.5, 256x1
//     34.4; 2048 180, 210; of 64 KB 304 rows 11.6, 11.4; 1024 35, 28; of 128 KB 2048
//     99, 96
//   rows above 320 KB over the fewest CTAs of 512 that keep a share below that, above
//     640 KB over twice as many of 256 (four rows' CTAs to an SM instead of two while
//     one waits for its peers).  1024 x 512 KB 512x2 197, 512x1 211, 512x4 224; 1024 x
//     1 MB 256x8 393, 512x4 402, 512x2 436, 512x1 457
// Kept in shared memory, of 2048 rows of 256 KB: nothing 190.6, 32 KB 185.7, 64 KB
// 182.7, 96 KB 180.2; what is left of L1 has to hold the loads in flight.
struct GradPlan {
  int threads, ctas, keep;
};
static GradPlan grad_plan(int32_t n, int64_t bytes) {
  if (bytes <= 16 * 1024) return {128, 1, 0};
  int c = 1;
  if ((n <= 64 && bytes >= 48 * 1024) || (n <= 128 && bytes >= 128 * 1024)) {
    const int most = bytes >= 128 * 1024 ? 512 : 256;
    while (c < kMaxCluster && n * c * 2 <= most && bytes / (2 * c) >= 15 * 1024) c *= 2;
    return {256, c, 2};
  }
  if (n > 2 * device_attr<cudaDevAttrMultiProcessorCount>() && bytes <= 160 * 1024) return {256, 1, 2};
  while (c < kMaxCluster && bytes / c > 320 * 1024) c *= 2;
  if (c == 4) return {256, 8, 2};
  return {512, c, c == 1 ? 3 : 2};
}

template <typename TIn, bool kEntropy, int T>
static ls_status launch_grad(const TokenArgs& a, ls_dtype dtype, const GradPlan& p, cudaStream_t st) {
  static std::atomic<int> done[kMaxDevices];
  const int upc = (int)((row_units(a.vocab, dtype) + p.ctas - 1) / p.ctas);
  if ((int64_t)a.n * p.ctas > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  auto kernel = token_grad_kernel<TIn, kEntropy, T>;
  if (!open_limits(kernel, done)) return LS_ERR_CUDA;
  const int stages = upc / (kStage * T), keep = p.keep < stages ? p.keep : stages;
  return launch_kernel(kernel, dim3((unsigned)a.n * p.ctas), T, p.ctas, (size_t)keep * kStage * T * 32, st, a, upc, keep);
}

template <typename TIn, bool kEntropy>
static ls_status pick_grad(const TokenArgs& a, ls_dtype dtype, const GradPlan& p, cudaStream_t st) {
  return p.threads == 128   ? launch_grad<TIn, kEntropy, 128>(a, dtype, p, st)
         : p.threads == 256 ? launch_grad<TIn, kEntropy, 256>(a, dtype, p, st)
                            : launch_grad<TIn, kEntropy, 512>(a, dtype, p, st);
}

ls_status token_grad(const TokenArgs& a, ls_dtype dtype, bool entropy, cudaStream_t st) {
  const GradPlan p = grad_plan(a.n, row_units(a.vocab, dtype) * 32);
  if (dtype == LS_DTYPE_BF16)
    return entropy ? pick_grad<bf16_tag, true>(a, dtype, p, st) : pick_grad<bf16_tag, false>(a, dtype, p, st);
  return entropy ? pick_grad<float, true>(a, dtype, p, st) : pick_grad<float, false>(a, dtype, p, st);
}

}  // namespace ops
}  // namespace lsg
