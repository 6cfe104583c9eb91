// Losses over a vocabulary in pieces, and their gradients (implemented in vocab.hip).
#pragma once

#include <vector>

#include "exec.h"

namespace ar {

constexpr double kLog2e = 1.4426950408889634;  // exponentials are powers of 2: of logits times this

enum Reduction : int32_t { R_MEAN = 0, R_SUM = 1, R_NONE = 2 };

// One rank's rows of the output matrix, and where their gradient goes.
struct VocabPiece {
  const void* w = nullptr;
  void* dw = nullptr;
  int64_t rows = 0, ld = 0, dld = 0;
};

// Arguments have been validated.
struct Vocab {
  int64_t T = 0, H = 0;
  int32_t dtype = 0;
  const void* hidden = nullptr;
  int64_t ld = 0;
  std::vector<VocabPiece> pieces;
  float temperature = 1;
  int32_t reduction = R_MEAN;
  const float* token_weights = nullptr;  // null: 1
  int32_t top = 0;                       // teacher's logits a row; 0: one target a row
  const void* ids = nullptr;             // targets [T], or teacher ids [T, top]
  bool wide_ids = true;                  // int64, or int32
  int64_t ids_ld = 0, ignore = -100;
  const void* logits = nullptr;  // teacher logits [T, top]
  int32_t logits_dtype = 0;
  int64_t logits_ld = 0;
  float* loss = nullptr;  // one value, or T
  void* dh = nullptr;
  int64_t dh_ld = 0;
  void* workspace = nullptr;
  size_t workspace_bytes = 0;
  void* start_event = nullptr;
  void* stop_event = nullptr;
};

RunResult run_vocab(const Vocab& v, bool grad, void* stream);
size_t vocab_workspace(const Vocab& v, bool grad);

}  // namespace ar
