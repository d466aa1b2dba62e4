// la_heads_common.h -- host-side checks of tensors of heads [tokens, heads, D] with a stride between
// tokens and one between heads (la_rotary.h, la_attention.h).
#pragma once

#include <cstdint>

#include "la_rows_common.h"

namespace la_host {

// A tensor of heads as the caller gave it.
struct HeadsArg {
  const void* p;
  int64_t ld, hs;
  int64_t tokens, heads;
  int D;
  uint64_t element, align;  // bytes; align also of the strides
  const char* name;
};

// The argument as given, with a stride of a single head or token, which addresses nothing, replaced.
inline HeadsArg heads_arg(const void* p, int64_t ld, int64_t hs, int64_t tokens, int64_t heads, int D, uint64_t element,
                          uint64_t align, const char* name) {
  if (heads == 1) hs = D;
  if (tokens == 1) ld = (heads - 1) * hs + D;
  return {p, ld, hs, tokens, heads, D, element, align, name};
}

// The span of a tensor of heads: rows of a token's heads, or (head-major) of a head's tokens.
inline RowSpan span_of(const HeadsArg& h) {
  const bool token_major = h.ld >= h.hs;
  const int64_t outer = token_major ? h.tokens : h.heads, inner = token_major ? h.heads : h.tokens;
  const int64_t so = token_major ? h.ld : h.hs, si = token_major ? h.hs : h.ld;
  if (h.tokens == 0) return {nullptr, 0, 0, 0, 1, 0, 0, h.name};
  return {h.p,     static_cast<uint64_t>((inner - 1) * si + h.D) * h.element, static_cast<uint64_t>(so) * h.element,
          static_cast<uint64_t>(outer), h.align, 0, 0, h.name};
}

// Strides that keep every element of the tensor apart, and alignment.
inline la_status check_heads(const HeadsArg& h) {
  if (!h.p || h.tokens == 0) return LA_OK;
  constexpr int64_t kMost = int64_t(1) << 40;
  const bool token_major = h.ld >= h.hs;
  const int64_t outer = token_major ? h.ld : h.hs, inner = token_major ? h.hs : h.ld;
  const int64_t n = token_major ? h.heads : h.tokens;
  if (outer > kMost || inner < h.D || outer < (n - 1) * inner + h.D)
    return fail(LA_ERR_INVALID_ARGUMENT, "the strides of %s (%lld between tokens, %lld between heads) do not keep its heads apart",
                h.name, (long long)h.ld, (long long)h.hs);
  if (reinterpret_cast<uintptr_t>(h.p) % h.align != 0)
    return fail(LA_ERR_INVALID_ARGUMENT, "%s must be %d-byte aligned", h.name, (int)h.align);
  if (h.align > h.element && (h.ld * h.element % h.align != 0 || h.hs * h.element % h.align != 0))
    return fail(LA_ERR_INVALID_ARGUMENT, "the strides of %s must be multiples of %d elements", h.name,
                (int)(h.align / h.element));
  return LA_OK;
}

// Outputs against inputs and against each other.
inline la_status check_apart(const RowSpan* ins, int n_in, const RowSpan* outs, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (share(outs[i], ins[j]))
        return fail(LA_ERR_INVALID_ARGUMENT, "%s overlaps %s (an output may share no memory with an input)",
                    outs[i].name, ins[j].name);
    for (int j = 0; j < i; ++j)
      if (share(outs[i], outs[j]))
        return fail(LA_ERR_INVALID_ARGUMENT, "%s overlaps %s (outputs may share no memory)", outs[i].name,
                    outs[j].name);
  }
  return LA_OK;
}

}  // namespace la_host
