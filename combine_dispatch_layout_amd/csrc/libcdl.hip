// libcdl.hip -- the library as one translation unit: the expert kernels, the
// products and the norm share the layout's device functions and the host-side argument
// checks of the dispatch/combine file.
#include "cdl.hip"
#include "experts.hip"
#include "products.hip"
#include "norm.hip"
