// The 8-bit product's tensor-core kernel (k_i8tc.cu), as its callers see it.
#pragma once
#include "os2_internal.cuh"

struct I8TcArgs {
  int m, n, k;                 // tokens, channels, terms (k >= 1)
  const void *tokens;          // FP16 integers [m][pitch], pitch a multiple of 8, 16-byte aligned
  long pitch;
  const void *W;               // int8 [n][ldw], ldw a multiple of 16, 16-byte aligned
  long ldw;
  const float *sa, *sb, *bias; // bias may be null
  void *y;
  long ldy;
  int out_dtype;
  int *slots;                  // I8TcSizes
  unsigned *done;              // zero before the launch
  int *status;
};
struct I8TcSizes {
  int counters;                // of `done`
  size_t slot_ints;
};
I8TcSizes i8tc_sizes(int m, int n, int k);
cudaError_t launch_i8tc(const I8TcArgs &a, cudaStream_t s);
