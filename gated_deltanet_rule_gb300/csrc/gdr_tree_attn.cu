// gdr_tree_attn: attention of drafted nodes over the pages (the kernels are in gdr_attn_frame.cuh).
#include "gdr_attn_frame.cuh"

namespace gdr {
namespace {

template <int D, int kForm>
cudaError_t launch_tree(const TreeAttnArgs& p, cudaStream_t st) {
  Args a{};
  a.B = p.B;
  return launch<D, kForm>(p, a, st);
}

template <int D>
cudaError_t launch_two(const TreeAttnArgs& a, cudaStream_t s) {
  // more nodes than one M tile holds: two M tiles share the key/value tiles' way through shared memory and
  // from HBM. What decides is whether the keys and values fit in L2, which the host cannot know (the contexts
  // are on the device). Where they do not, kWide is far ahead (heads of 64, then of 128; kWide and kNarrow):
  // 16 rows of 17 nodes over up to 32768 positions, 32 / 4 heads 123 and 150, 142 and 222 us; 8 rows of 64
  // nodes over 65536, 32 / 8 heads 246 and 343, 290 and 456; 8 rows of 64 nodes over 16384, 32 / 4 heads of 128
  // 95 and 111. Where they do, kNarrow is ahead by up to a fifth: 8 rows of 17 and of 32 nodes over 8192, 32 / 4
  // heads 39.0 and 34.9, 43.0 and 39.7 us, and 44.5 and 35.2, 49.4 and 41.6; a prefill chain of 2048 by 4%.
  return a.N > kM / (a.Hq / a.Hk) ? launch_tree<D, kWide>(a, s) : launch_tree<D, kNarrow>(a, s);
}

}  // namespace

size_t tree_attn_workspace_bytes(int D) { return parts_bytes(D); }

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t s) {
  return a.D == 64 ? launch_two<64>(a, s) : a.D == 128 ? launch_two<128>(a, s) : launch_tree<256, kSplit>(a, s);
}

}  // namespace gdr
