// What the join may take from the workspace.  A CTA of the chunk kernel that
// gave up on a wait leaves the entries of its cut units unwritten, and a
// workspace may hold anything: an entry is used only if it names a unit of this
// call, cut into as many parts as the call cuts its units into (that number is
// written before any wait).  Then every address made from it lies inside the
// call's tensors and workspace.  Host code too, so that it is tested there.
#pragma once

#ifdef __CUDACC__
#define SINK_ATTN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SINK_ATTN_HOST_DEVICE inline
#endif

namespace sa {

// An entry {request, unit within its head, head, parts}; rows(b): tokens of
// request b, 0 if none of them are in units of `unit` tokens, which may be
// asked for once b is known to be a request.  (A product, not a division: the
// join's CTAs do little else than wait, and a division took them 1 us of 49.)
template <typename Rows>
SINK_ATTN_HOST_DEVICE bool cut_unit_fits(int b, int group, int head, int parts, int batch, int heads, int call_parts,
                                         int unit, Rows rows) {
  return b >= 0 && b < batch && head >= 0 && head < heads && parts == call_parts && group >= 0 &&
         static_cast<long long>(group) * unit < rows(b);
}

}  // namespace sa
