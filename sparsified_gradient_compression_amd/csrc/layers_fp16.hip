// layers_fp16.hip -- the layer operators' kernels for fp16 elements.
#include "layers_launch.hpp"

template struct dgc::layers::Launch<_Float16>;
