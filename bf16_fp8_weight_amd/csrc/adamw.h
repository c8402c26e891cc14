// adamw.h -- the AdamW step's tables (shared by the host builder and the
// kernels) and its host-only builder: validation of the tensor table and the
// work list. Nothing declared here calls the HIP runtime.
#pragma once

#include <cstdint>
#include <string>
#include <vector>

#include "wt.h"

namespace wt {

constexpr int kAdamBlock = 128;   // elements that share one scale of an 8-bit state
// Elements of one work item (one workgroup, eight to a thread). Measured on
// MI355X over 176 M elements: 32-bit states 880 / 848 / 942 us with 256 / 512 /
// 1024 threads, 8-bit states 470 / 497 us with 256 / 512 (their registers).
constexpr int adam_item(int state_bits) { return state_bits == 32 ? 4096 : 2048; }
constexpr int kAdamNormGrid = 2048;  // most workgroups of the norm kernel (one partial sum each)

enum : uint32_t {
  kAdamGradBf16 = 1,
  kAdamMaster = 2,
  kAdamParam = 4,
  // every 4-element chunk of every array starts at its vector access's alignment; one array that does not sends all of
  // the tensor's through 1-, 2- and 4-byte accesses (176 M elements, BF16 shards at odd elements: 32-bit states 852 ->
  // 1467 us, 8-bit 493 -> 1099 us)
  kAdamVector = 8,
};

// One tensor of the step; addresses as integers.
struct AdamTensor {
  uint64_t param, master, grad, m, v, m_scale, v_scale;
  int64_t n;
  uint32_t block0;  // number of the tensor's first 128-element block in the table
  uint32_t flags;
  float lr_mul;
  float weight_decay;
};
static_assert(sizeof(AdamTensor) == 80, "AdamTensor layout");

// Elements [item chunk, item (chunk + 1)) of one tensor.
struct AdamItem {
  uint32_t tensor;
  uint32_t chunk;
};

// The same elements as the norm kernel reads them, address resolved.
struct AdamGradItem {
  uint64_t grad;   // address of the item's first gradient
  uint32_t count;  // elements
  uint32_t flags;  // of the tensor
};

// The step's scalars as the kernels use them.
struct AdamScalars {
  float lr;          // learning rate
  float lr_bias1;    // lr / (1 - beta1^t)
  float b1, ib1;     // beta1, 1 - beta1
  float b2, ib2;
  float inv_bias2;   // 1 / sqrt(1 - beta2^t)
  float eps;
  uint32_t k0, k1;   // keys of the step's random bits
};

// What the update kernel takes from the norm.
struct AdamNorm {
  float clip;
  uint32_t skip;  // the norm is not finite: the step changes nothing
};

struct AdamLayout {
  std::vector<AdamTensor> tensors;  // those with elements
  std::vector<AdamItem> items;
  std::vector<AdamGradItem> grads;  // one per item
  int32_t state_bits = 32;
  wt_adamw_info info{};
};

// Byte offsets of the parts of a handle's one device allocation.
struct AdamOffsets {
  uint64_t tensors, items, grads, partials, norm, bytes;
};
AdamOffsets adamw_offsets(const AdamLayout &L);

wt_adamw_options resolve_adamw_opts(const wt_adamw_options *o);
wt_status build_adamw(const wt_adamw_tensor *t, size_t n, const wt_adamw_options &o, AdamLayout *L, std::string *err);

// Checks hyper values; the text says what is out of range.
wt_status check_adamw_hyper(const wt_adamw_hyper *h, std::string *err);

}  // namespace wt
