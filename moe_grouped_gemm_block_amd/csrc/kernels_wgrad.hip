// Definitions of the weight gradient's kernels.
#define DG_DEFINE_WGRAD
#include "wgrad.hpp"
