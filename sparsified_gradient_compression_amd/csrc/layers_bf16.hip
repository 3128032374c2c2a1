// layers_bf16.hip -- the layer operators' kernels for bf16 elements.
#include "layers_launch.hpp"

template struct dgc::layers::Launch<__bf16>;
