// The join of a block with its residual stream: which kernel a call takes
// (residual_kernels.cuh).
#include "residual_kernels.cuh"

namespace mok {

namespace residual {

#define MOK_RESIDUAL_INSTANCES(S, B)                                                                    \
  extern template cudaError_t forward_rows<S, B, true>(const ResidualParams&, cudaStream_t);            \
  extern template cudaError_t forward_rows<S, B, false>(const ResidualParams&, cudaStream_t);           \
  extern template cudaError_t backward_rows<S, B, true>(const ResidualParams&, int*, cudaStream_t);     \
  extern template cudaError_t backward_rows<S, B, false>(const ResidualParams&, int*, cudaStream_t);
MOK_RESIDUAL_INSTANCES(__nv_bfloat16, __nv_bfloat16)
MOK_RESIDUAL_INSTANCES(float, __nv_bfloat16)
MOK_RESIDUAL_INSTANCES(float, float)

namespace {

template <typename E>
bool vectors(const void* ptr, long ld) {
  return !ptr || (reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld % (16 / (int)sizeof(E)) == 0);
}

// Whether every row of every tensor is made of whole 16-byte vectors.
template <typename S, typename B>
bool all_vectors(const ResidualParams& p) {
  return p.H % 8 == 0 && vectors<B>(p.w_out, 0) && vectors<B>(p.gate, 0) && vectors<B>(p.w_next, 0) &&
         vectors<S>(p.x, p.ldx) && vectors<B>(p.y, p.ldy) && vectors<S>(p.xo, p.ldxo) && vectors<B>(p.n, p.ldn) &&
         vectors<S>(p.dxo, p.lddxo) && vectors<B>(p.dn, p.lddn) && vectors<S>(p.dx, p.lddx) &&
         vectors<B>(p.dy, p.lddy) && vectors<B>(p.dgate, 0);
}

template <typename S, typename B>
cudaError_t any_forward(const ResidualParams& p, cudaStream_t st) {
  return all_vectors<S, B>(p) ? forward_rows<S, B, true>(p, st) : forward_rows<S, B, false>(p, st);
}
template <typename S, typename B>
cudaError_t any_backward(const ResidualParams& p, int* launches, cudaStream_t st) {
  return all_vectors<S, B>(p) ? backward_rows<S, B, true>(p, launches, st) : backward_rows<S, B, false>(p, launches, st);
}

}  // namespace
}  // namespace residual

size_t residual_part_floats(int T, int H) {
  using namespace residual;
  // (units are no more than workers where their sums are parts)
  size_t most = 0;
  for (const bool aligned : {false, true}) {
    const int ng = groups_backward(H, aligned), nt = team_threads(H, ng), rows = nt == 32 ? kTeamRows : 1;
    const BackwardPlan b = backward_plan(T, 0, device_sm_count() * ctas_backward(nt * rows, ng) * rows, rows);
    most = std::max(most, (2 * (size_t)b.ctas + b.workers) * H);
  }
  return most;
}

cudaError_t launch_residual_forward(mok_dtype stream, mok_dtype branch, const ResidualParams& p, int* launches,
                                    cudaStream_t st) {
  *launches = 1;
  if (stream == MOK_TYPE_BF16) return residual::any_forward<__nv_bfloat16, __nv_bfloat16>(p, st);
  return branch == MOK_TYPE_BF16 ? residual::any_forward<float, __nv_bfloat16>(p, st) : residual::any_forward<float, float>(p, st);
}

cudaError_t launch_residual_backward(mok_dtype stream, mok_dtype branch, const ResidualParams& p, int* launches,
                                     cudaStream_t st) {
  if (stream == MOK_TYPE_BF16) return residual::any_backward<__nv_bfloat16, __nv_bfloat16>(p, launches, st);
  return branch == MOK_TYPE_BF16 ? residual::any_backward<float, __nv_bfloat16>(p, launches, st)
                                 : residual::any_backward<float, float>(p, launches, st);
}

}  // namespace mok
